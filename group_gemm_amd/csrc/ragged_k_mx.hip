// ragged_k_mx.hip -- contracting ragged dot (the weight-gradient case) from rows kept in MXFP8, gfx950:
//   out[h] = alpha * value(lhs[rows of h, :])^T . dout[rows of h, :] + beta * out[h]      -> out [g, k, n]
// with lhs e4m3 codes [m, k], one E8M0 scale per 32 along k, and dout bf16.
//
// A scale belongs to one row, and rows are what is contracted, so no matrix instruction can apply it: the codes are
// turned to bf16 (which holds every value of them) on their way into LDS, 32 of a row's codes and one scale a
// thread, and the product is the bf16 one.  Both tiles have the contracted rows as their slow axis and are read with
// ds_read_b64_tr_b16 into row-consecutive fragments.  Groups longest first, as in ragged_k.hip.
#include "common.hpp"
#include "launch.hpp"

namespace gg {
namespace kmx {

constexpr int BM = 256, BN = 256, BR = 64, NT = 512;   // BM along k (output rows), BN along n
constexpr int LPT_MAX_G = 64;                           // longest-first order up to this many groups
typedef i32x4 __attribute__((aligned(2))) i32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

struct Smem {
    uint16_t a[2][BR * BM];
    uint16_t b[2][BR * BN];
    Tables tab;
    int order[LPT_MAX_G];
};

// row-major [64][256] with 16-byte pieces XOR'ed in 64-byte units by a 3-bit function of the row, so the rows that
// one transposing read touches lie in distinct banks
__device__ inline int swz(int r) { return ((r & 3) | (((r >> 3) & 1) << 2)) << 2; }
__device__ inline int off(int r, int c) { return r * 256 + (((c >> 3) ^ swz(r)) << 3) + (c & 7); }

// what a thread holds of the next 64 rows: 32 codes of row t / 8 with their scale, and eight columns of dout's rows
// t / 32 + 16 i
struct Regs { i32x4 a[2]; int byte; i32x4 b[4]; };

__device__ inline void load(Regs& v, const KmxParams& p, int row0, int rows, int i0, int j0) {
    const int t = threadIdx.x;
    const int r = t >> 3, c = i0 + 32 * (t & 7);
    v.a[0] = v.a[1] = i32x4{0, 0, 0, 0};
    v.byte = 0;
    if (r < rows && c < p.k) {
        const i32x4* at = (const i32x4*)(p.lhs + (int64_t)(row0 + r) * p.k + c);
        v.a[0] = at[0];
        v.a[1] = at[1];
        v.byte = p.lhs_scale[(int64_t)(row0 + r) * (p.k >> 5) + (c >> 5)];
    }
    const int n0 = j0 + 8 * (t & 31);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = (t >> 5) + 16 * i;
        v.b[i] = i32x4{0, 0, 0, 0};
        if (q >= rows || n0 >= p.n) continue;
        const uint16_t* at = p.dout + (int64_t)(row0 + q) * p.n + n0;
        if (n0 + 8 <= p.n) v.b[i] = *(const i32x4_any*)at;
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n0 + e < p.n) v.b[i][e >> 1] |= (int)((uint32_t)at[e] << (16 * (e & 1)));
        }
    }
}
__device__ inline void store(const Regs& v, uint16_t* a, uint16_t* b) {
    const int t = threadIdx.x;
    const float s = __uint_as_float((uint32_t)v.byte << 23);   // exponent field 255 is NaN to the conversion
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        i32x4 q;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const uint32_t c = (uint32_t)v.a[i >> 1][2 * (i & 1) + d];
            q[2 * d] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false));
            q[2 * d + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true));
        }
        *(i32x4*)(a + off(t >> 3, 32 * (t & 7) + 8 * i)) = q;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) *(i32x4*)(b + off((t >> 5) + 16 * i, 8 * (t & 31))) = v.b[i];
}

// rows 16 s + 8 (l / 32) .. + 7 of column col0 + l % 32
__device__ inline bf16x8 frag(const uint16_t* tile, int s, int col0) {
    const int l = threadIdx.x & 63, q = l >> 4;
    const int c = col0 + 16 * (q & 1) + 4 * (l & 3), r = 16 * s + 8 * (q >> 1) + ((l >> 2) & 3);
    const i16x4 lo = lds_read_tr16(tile + off(r, c)), hi = lds_read_tr16(tile + off(r + 4, c));
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
}

__device__ inline float get(const float* p) { return *p; }
__device__ inline float get(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ inline void put(float* p, float v) { *p = v; }
__device__ inline void put(uint16_t* p, float v) { const __bf16 b = (__bf16)v; *p = __builtin_bit_cast(uint16_t, b); }

template <typename O>
__global__ __launch_bounds__(NT, 1) void kernel(KmxParams p) {
    __shared__ Smem sm;
    const int t = threadIdx.x, wave = t >> 6, wm = wave >> 2, wn = wave & 3, l = t & 63;
    const int nti = cdiv(p.k, BM), ntj = cdiv(p.n, BN), per = nti * ntj, total = p.g * per;
    const bool lpt = p.g <= LPT_MAX_G;
    int gemm_tiles, covered;
    build_tables<NT>(p.group_sizes, p.g, p.m, 1, 0, sm.tab, &gemm_tiles, &covered);
    if (blockIdx.x == 0 && t == 0) *p.status = sm.tab.flags;
    if (lpt) {   // rank of every group by (size desc, index asc)
        if (t < p.g) {
            const int st = sm.tab.row_off[t + 1] - sm.tab.row_off[t];
            int rank = 0;
            for (int j = 0; j < p.g; ++j) {
                const int sj = sm.tab.row_off[j + 1] - sm.tab.row_off[j];
                rank += (sj > st) || (sj == st && j < t);
            }
            sm.order[rank] = t;
        }
        __syncthreads();
    }
    for (int tile = xcd_virtual_id(blockIdx.x, gridDim.x); tile < total; tile += gridDim.x) {
        const int pg = tile / per, local = tile - pg * per, grp = lpt ? sm.order[pg] : pg;
        const int row0 = sm.tab.row_off[grp], size = sm.tab.row_off[grp + 1] - row0;
        const int i0 = (local % nti) * BM, j0 = (local / nti) * BN;
        f32x16 acc[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
        Regs v;
        if (size > 0) {
            load(v, p, row0, size, i0, j0);
            store(v, sm.a[0], sm.b[0]);
            __syncthreads();
        }
        int slot = 0;
        for (int r = 0; r < size; r += BR, slot ^= 1) {
            const bool more = r + BR < size;
            if (more) load(v, p, row0 + r + BR, size - r - BR, i0, j0);
#pragma unroll
            for (int s = 0; s < BR / 16; ++s) {
                bf16x8 a[4], b[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = frag(sm.a[slot], s, 128 * wm + 32 * i);
#pragma unroll
                for (int j = 0; j < 2; ++j) b[j] = frag(sm.b[slot], s, 64 * wn + 32 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
            }
            if (more) store(v, sm.a[slot ^ 1], sm.b[slot ^ 1]);
            __syncthreads();
        }
        O* out = (O*)p.out + (int64_t)grp * p.k * p.n;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int r = i0 + 128 * wm + 32 * i + 8 * (e >> 2) + 4 * (l >> 5) + (e & 3), c = j0 + 64 * wn + 32 * j + (l & 31);
                    if (r >= p.k || c >= p.n) continue;
                    O* at = out + (int64_t)r * p.n + c;
                    float x = p.alpha * acc[i][j][e];
                    if (p.beta != 0.f) x += p.beta * get(at);
                    put(at, x);
                }
    }
}

}  // namespace kmx

hipError_t launch_ragged_k_mx(const KmxParams& p, int grid, hipStream_t s) {
    if (p.out_f32) hipLaunchKernelGGL(kmx::kernel<float>, dim3(grid), dim3(kmx::NT), 0, s, p);
    else hipLaunchKernelGGL(kmx::kernel<uint16_t>, dim3(grid), dim3(kmx::NT), 0, s, p);
    return hipGetLastError();
}

}  // namespace gg
