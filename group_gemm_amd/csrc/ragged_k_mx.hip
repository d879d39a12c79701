// ragged_k_mx.hip -- contracting ragged dot (the weight-gradient case) from rows kept in MXFP8, gfx950:
//   out[h] = alpha * value(lhs[rows of h, :])^T . dout[rows of h, :] + beta * out[h]      -> out [g, k, n]
// with lhs e4m3 codes [m, k], one E8M0 scale per 32 along k, and dout bf16.
//
// A scale belongs to one row, and rows are what is contracted, so no matrix instruction can apply it: the codes are
// turned to bf16 (which holds every value of them) on their way into LDS, 32 of a row's codes and one scale a
// thread, and the product is the bf16 one.  Both tiles have the contracted rows as their slow axis and are read with
// ds_read_b64_tr_b16 into row-consecutive fragments.  Groups longest first, as in ragged_k.hip.
//
// Two kernels: the ring one below for n a multiple of 8 and 16-byte aligned operands, the general one for the rest.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "ring.hpp"

namespace gg {

// With few tiles a group's rows are dealt to `splits` workgroups in runs of whole 32-row slices; their results are added
// up in order by kmx::add_up.
__device__ inline void part_of(int splits, int part, int& row0, int& size) {
    if (splits == 1) return;
    const int run = cdiv(cdiv(size, splits), 32) * 32, at = (int)min((int64_t)part * run, (int64_t)size);
    row0 += at;
    size = min(run, size - at);
}

namespace kmx {

constexpr int BN = 256, NT = 512;   // a tile is 64 MI x 256 of k x n (MI 4, or 2 for few rows), BR rows a step
constexpr int LPT_MAX_G = 64;                           // longest-first order up to this many groups
typedef i32x4 __attribute__((aligned(2))) i32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

constexpr int SP = 64 + 4;
template <int BR, int SLOTS> struct Smem {
    union {
        struct { uint16_t a[SLOTS][BR * 256], b[SLOTS][BR * BN]; };
        float strips[8][32 * SP];
    };
    Tables tab;
    int order[LPT_MAX_G];
};

// row-major [BR][256] with 16-byte pieces XOR'ed in 64-byte units by a 3-bit function of the row, so the rows that
// one transposing read touches lie in distinct banks
__device__ inline int swz(int r) { return ((r & 3) | (((r >> 3) & 1) << 2)) << 2; }
__device__ inline int off(int r, int c) { return r * 256 + (((c >> 3) ^ swz(r)) << 3) + (c & 7); }

// what a thread holds of the next BR rows: 32 codes of row t / 8 with their scale, and eight columns of dout's rows
// t / 32 + 16 i
template <int BR> struct Regs { i32x4 a[2]; int byte; i32x4 b[BR / 16]; };

template <int BR>
__device__ inline void load(Regs<BR>& v, const KmxParams& p, int row0, int rows, int i0, int i1, int j0) {
    const int t = threadIdx.x;
    const int r = t >> 3, c = i0 + 32 * (t & 7);
    v.a[0] = v.a[1] = i32x4{0, 0, 0, 0};
    v.byte = 0;
    if (r < min(rows, BR) && c < i1) {
        const i32x4* at = (const i32x4*)(p.lhs + (int64_t)(row0 + r) * p.k + c);
        v.a[0] = at[0];
        v.a[1] = at[1];
        v.byte = p.lhs_scale[(int64_t)(row0 + r) * (p.k >> 5) + (c >> 5)];
    }
    const int n0 = j0 + 8 * (t & 31);
#pragma unroll
    for (int i = 0; i < BR / 16; ++i) {
        const int q = (t >> 5) + 16 * i;
        v.b[i] = i32x4{0, 0, 0, 0};
        if (q >= rows || n0 >= p.n) continue;
        const uint16_t* at = p.dout + (int64_t)(row0 + q) * p.n + n0;
        if (at + 8 <= p.dout + (int64_t)p.m * p.n) {   // what lies behind the row is masked later, so that no load waits
            v.b[i] = *(const i32x4_any*)at;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n0 + e < p.n) v.b[i][e >> 1] |= (int)((uint32_t)at[e] << (16 * (e & 1)));
        }
    }
}
template <int BR>
__device__ inline void store(const Regs<BR>& v, uint16_t* a, uint16_t* b, int cols) {   // cols: dout's left, from the tile's first
    const int t = threadIdx.x;
    const float s = __uint_as_float((uint32_t)v.byte << 23);   // exponent field 255 is NaN to the conversion
    if (t < 8 * BR)
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
    for (int i = 0; i < BR / 16; ++i) {
        i32x4 q = v.b[i];
#pragma unroll
        for (int d = 0; d < 4; ++d) q[d] &= 8 * (t & 31) + 2 * d + 2 <= cols ? -1 : 8 * (t & 31) + 2 * d + 1 == cols ? 0xffff : 0;
        *(i32x4*)(b + off((t >> 5) + 16 * i, 8 * (t & 31))) = q;
    }
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
// (stores that the caches may hold back: a row of odd length shares its first and last line with its neighbours, and with
// the nontemporal hint each part went out by itself, 161 instead of 81 us for 32 groups of 12 rows, k 2880, n 1447)
__device__ inline void put8(float* p, const float (&v)[8]) {
    *(f32x4_any*)p = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4_any*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ inline void put8(uint16_t* p, const float (&v)[8]) {
    *(i32x4_any*)p = i32x4{(int)ring::pack_bf16(v[0], v[1]), (int)ring::pack_bf16(v[2], v[3]), (int)ring::pack_bf16(v[4], v[5]),
                           (int)ring::pack_bf16(v[6], v[7])};
}
__device__ inline void put(uint16_t* p, float v) { const __bf16 b = (__bf16)v; *p = __builtin_bit_cast(uint16_t, b); }

template <typename O, int MI, int BR, int SLOTS>
__global__ __launch_bounds__(NT, MI == 2 ? 4 : 1) void kernel(KmxParams p) {
    constexpr int BM = 64 * MI;
    __shared__ Smem<BR, SLOTS> sm;
    const int t = threadIdx.x, wave = t >> 6, wm = wave >> 2, wn = wave & 3, l = t & 63;
    const int nti = cdiv(p.k, BM), ntj = cdiv(p.n, BN), per = nti * ntj, total = p.g * p.splits * per;
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
        const int vg = tile / per, local = tile - vg * per, pg = vg / p.splits, part = vg - pg * p.splits, grp = lpt ? sm.order[pg] : pg;
        int row0 = sm.tab.row_off[grp], size = sm.tab.row_off[grp + 1] - row0;
        part_of(p.splits, part, row0, size);
        const int i0 = (local % nti) * BM, j0 = (local / nti) * BN;
        f32x16 acc[MI][2];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
        Regs<BR> v;
        if (size > 0) {
            load(v, p, row0, size, i0, min(p.k, i0 + BM), j0);
            store(v, sm.a[0], sm.b[0], p.n - j0);
            __syncthreads();
        }
        int slot = 0;
        for (int r = 0; r < size; r += BR, slot ^= SLOTS - 1) {
            const bool more = r + BR < size;
            if (more) load(v, p, row0 + r + BR, size - r - BR, i0, min(p.k, i0 + BM), j0);
#pragma unroll
            for (int s = 0; s < BR / 16; ++s) {
                bf16x8 a[MI], b[2];
#pragma unroll
                for (int i = 0; i < MI; ++i) a[i] = frag(sm.a[slot], s, 32 * MI * wm + 32 * i);
#pragma unroll
                for (int j = 0; j < 2; ++j) b[j] = frag(sm.b[slot], s, 64 * wn + 32 * j);
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
            }
            if (SLOTS == 1) __syncthreads();
            if (more) store(v, sm.a[slot ^ (SLOTS - 1)], sm.b[slot ^ (SLOTS - 1)], p.n - j0);
            __syncthreads();
        }
        // results turn in LDS, a strip of 32 x 64 a wave, and leave as whole row segments of 128 or 256 bytes, at any
        // alignment
        O* out = (O*)p.out + ((int64_t)grp * p.splits + part) * p.k * p.n;
        float* strip = sm.strips[wave];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    *(f32x4*)(strip + (l & 31) * SP + 32 * j + 8 * q + 4 * (l >> 5)) = v;
                }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int row = 8 * u + (l >> 3), r = i0 + 32 * MI * wm + 32 * i + row, c = j0 + 64 * wn + 8 * (l & 7);
                const f32x4 lo = *(const f32x4*)(strip + row * SP + 8 * (l & 7)), hi = *(const f32x4*)(strip + row * SP + 8 * (l & 7) + 4);
                if (r >= p.k || c >= p.n) continue;
                O* at = out + (int64_t)r * p.n + c;
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) { x[e] = p.alpha * lo[e]; x[4 + e] = p.alpha * hi[e]; }
                const int valid = min(8, p.n - c);
                if (p.beta != 0.f) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < valid) x[e] += p.beta * get(at + e);
                }
                if (valid == 8) put8(at, x);
                else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < valid) put(at + e, x[e]);
                }
            }
        }
        __syncthreads();   // the strips share memory with the tiles
    }
}

// out[h] = alpha * (sum of its parts) + beta * out[h]; V consecutive values a thread
template <typename O, int V>
__global__ __launch_bounds__(256) void add_up(const float* __restrict__ parts, O* __restrict__ out, int64_t per, int splits, float alpha,
                                              float beta) {
    const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (e >= per) return;
    const float* from = parts + (int64_t)blockIdx.y * splits * per + e;
    O* to = out + (int64_t)blockIdx.y * per + e;
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 0.f;
    for (int z = 0; z < splits; z += 4) {   // four parts' loads at a time, added in order
        float f[4][V];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float* at = from + (int64_t)min(z + u, splits - 1) * per;
            if constexpr (V == 4) {
                const f32x4 q = *(const f32x4_any*)at;
#pragma unroll
                for (int i = 0; i < V; ++i) f[u][i] = q[i];
            } else {
                f[u][0] = *at;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] += z + u < splits ? f[u][i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) put(to + i, alpha * s[i] + (beta != 0.f ? beta * get(to + i) : 0.f));
}

}  // namespace kmx

// The ring kernel: that of ragged_k_bf16.hip (a 256 x 256 tile a workgroup, four waves of 128 x 128, 32-row slices in a 4-slot
// LDS ring filled by loads straight into LDS, two pinned half-slice phases, groups longest first, 4 x 8 super-tiles), with
// the codes and their scales in a ring of their own.  A wave loads eight rows of a slice's codes (two loads) and their scales
// (one) and turns them itself, during the first half of the iteration before the one that multiplies them: its own loads are
// what it waits for, and the barrier that the iteration has anyway shows the bf16 slice to the other waves.  That is 16
// conversions, four LDS reads and four writes a wave beside 32 matrix instructions.
// Bound by the matrix instructions: 16384 rows of 16 groups, k 5120, n 8192, fp32 out, 1537 us or 895 TFLOP/s with groups of
// one size (the bf16 kernel 1410 to 1465) and 1605 with uneven ones, whose 2.7 GB of output alone take 550 at a copy's rate.
namespace kmxr {
using namespace ring;

constexpr int BM = 256, BN = 256, BR = 32, NT = 256, STAGES = 4;   // BM along k (output rows), BN along n
constexpr int MI = 4, NJ = 4, WCOLS = 128;
constexpr int SLICE = BR * 256;          // elements of one operand slice
constexpr int FIRST = 4, SECOND = 3;     // ring loads a thread: two of codes, one of scales, one of dout; three of dout
constexpr int PER = FIRST + SECOND;
constexpr int LPT_MAX_G = 256;           // longest-first order up to this many groups (O(g^2) ranking)
constexpr int SJ = 8;                    // n-tiles per super-tile column
static_assert(PER * (STAGES - 1) <= 63, "vmcnt range");

// one byte a lane, as a dword, straight into LDS at lds_addr + 4 * lane (ring.hpp)
__device__ inline void load_lds1(i32x4 r, uint32_t lds_addr, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_ubyte %1, %2, 0 offen lds"
                 :: "s"(lds_addr), "v"(off), "s"(r) : "memory", "m0");
}

struct Smem {
    struct {
        uint16_t b[STAGES][SLICE];
        uint16_t a[2][SLICE];
        uint8_t codes[STAGES][SLICE];
        uint32_t scale[STAGES][4][64];   // a wave's 8 rows of 8 scale bytes, one a dword
    } ring;
    Tables tab;
    int order[LPT_MAX_G];
};

// slice [32 rows][256 columns] as in ragged_k_bf16.hip
__device__ inline int swz(int kr) { return ((kr & 3) | (((kr >> 3) & 1) << 2)) << 2; }
__device__ inline int off(int kr, int nn) { return kr * 256 + (((nn >> 3) ^ swz(kr)) << 3) + (nn & 7); }

struct Frags { bf16x8 a[MI]; bf16x8 b[NJ]; };

// columns c0 + 32 j + (lane & 31), rows 16 s + 8 (lane / 32) .. + 7 of a slice
__device__ inline bf16x8 frag(const uint16_t* sl, int s, int c0, int j) {
    const int l = threadIdx.x & 63, q = l >> 4, rr = (l >> 2) & 3, c = l & 3;
    const int kr0 = 16 * s + 8 * (q >> 1) + rr;
    const int nn = c0 + 32 * j + 16 * (q & 1) + 4 * c;
    const i16x4 lo = lds_read_tr16(sl + off(kr0, nn));
    const i16x4 hi = lds_read_tr16(sl + off(kr0 + 4, nn));
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
}
// read number R of a step, in the order the MFMAs (column block major) first need them
template <int NB, int R>
__device__ inline void read_one(Frags& f, const uint16_t* a, const uint16_t* b, int s, int r0w, int c0w) {
    if constexpr (R >= 1 && R <= NB) f.a[R - 1] = frag(a, s, r0w, R - 1);
    else f.b[R == 0 ? 0 : R - NB] = frag(b, s, c0w, R == 0 ? 0 : R - NB);
}

// A lane's 32 codes of a slice on their way to bf16: the 16 it loaded of rows 8 wave + l / 16 and + 4 each.
struct Turn { i32x4 c[2]; uint32_t byte[2]; i32x4 v[4]; };

template <bool EPI, typename OutT, bool REBASE>
__global__ __launch_bounds__(NT, 1) void kernel(KmxParams p) {
    __shared__ Smem sm;
    const int t = threadIdx.x, l = t & 63, wave = t >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int r0w = 128 * wm, c0w = 128 * wn;   // wave's sub-tile: output rows (k) r0w.., columns (n) c0w..
    const int nti = cdiv(p.k, BM), ntj = cdiv(p.n, BN);
    const int per = nti * ntj;
    const int total = p.g * p.splits * per;
    const bool lpt = p.g <= LPT_MAX_G;
    int gemm_tiles, covered;
    build_tables<NT>(p.group_sizes, p.g, p.m, 1, 0, sm.tab, &gemm_tiles, &covered);
    if (blockIdx.x == 0 && t == 0) *p.status = sm.tab.flags;
    if (lpt) {   // rank of every group by (size desc, index asc)
        for (int h = t; h < p.g; h += NT) {
            const int sh = sm.tab.row_off[h + 1] - sm.tab.row_off[h];
            int rank = 0;
            for (int j = 0; j < p.g; ++j) {
                const int sj = sm.tab.row_off[j + 1] - sm.tab.row_off[j];
                rank += (sj > sh) || (sj == sh && j < h);
            }
            sm.order[rank] = h;
        }
        __syncthreads();
    }
    const uint32_t k1 = (uint32_t)p.k, ks = (uint32_t)p.k >> 5, n2 = (uint32_t)p.n * 2u;
    constexpr int osz = sizeof(OutT);

    // ring-load roles.  dout: slice [32 rows][256 cols] in 1 KiB blocks of 2 rows; wave w fills blocks 4 w + u; lane l writes
    // physical chunk l % 32 of row 2 (4 w + u) + l / 32, which holds logical chunk (l & 31) ^ swz(row).  Codes: load u of
    // wave w is rows 8 w + 4 u .. + 3, lane l the 16 codes at 16 (l % 16) of row l / 16.  Scales: lane l byte l % 8 of row
    // 8 w + l / 8.
    const int wave_u = __builtin_amdgcn_readfirstlane(wave);
    int ch8[4];
    uint32_t b_lane[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = 2 * (4 * wave + u) + (l >> 5);
        ch8[u] = 8 * ((l & 31) ^ swz(row));
        b_lane[u] = (uint32_t)(l >> 5) * n2 + (uint32_t)ch8[u] * 2u;
    }
    const uint32_t a_lane = (uint32_t)(l >> 4) * k1 + 16u * (uint32_t)(l & 15);
    const uint32_t s_lane = (uint32_t)(l >> 3) * ks + (uint32_t)(l & 7);
    const uint32_t lds_b = lds_u32(&sm.ring.b[0][0]) + (uint32_t)(4 * wave_u) * 1024u;
    const uint32_t lds_c = lds_u32(&sm.ring.codes[0][0]) + (uint32_t)wave_u * 2048u;
    const uint32_t lds_s = lds_u32(&sm.ring.scale[0][0][0]) + (uint32_t)wave_u * 256u;

    for (int tile = xcd_virtual_id(blockIdx.x, gridDim.x); tile < total; tile += gridDim.x) {
        const int vg = tile / per;
        int local = tile - vg * per;
        const int pg = vg / p.splits, part = vg - pg * p.splits, grp = lpt ? sm.order[pg] : pg;
        int row_base = sm.tab.row_off[grp], size = sm.tab.row_off[grp + 1] - row_base;
        part_of(p.splits, part, row_base, size);
        // (k-tile, n-tile) in super-tiles of SJ n-tiles
        const int full_sc = ntj / SJ;
        int it, jt;
        if (local < full_sc * SJ * nti) {
            const int sc = local / (SJ * nti), lo = local - sc * SJ * nti;
            it = lo / SJ; jt = sc * SJ + lo % SJ;
        } else {
            const int wl = ntj - full_sc * SJ, lo = local - full_sc * SJ * nti;
            it = lo / wl; jt = full_sc * SJ + lo % wl;
        }
        const int i0 = it * BM, j0 = jt * BN;
        const int rows_valid = min(BM, p.k - i0);   // output rows of the tile
        const int nb = max(0, min(MI, cdiv(rows_valid - r0w, 32)));
        const int nk = cdiv(size, BR);

        // Descriptors: with REBASE each covers one 32-row slice (its rows of the group), otherwise the group's rows (all of
        // lhs and dout span less than 2 GiB).  Either way rows past the group, and slices past its end, read as zeros into
        // slots that no one multiplies.
        struct SliceRsrc { i32x4 a, s, b; };
        const SliceRsrc group_rs = REBASE ? SliceRsrc{} : SliceRsrc{
            make_rsrc_v(p.lhs + (size_t)row_base * p.k, (uint32_t)size * k1),
            make_rsrc_v(p.lhs_scale + (size_t)row_base * ks, (uint32_t)size * ks),
            make_rsrc_v(p.dout + (size_t)row_base * p.n, (uint32_t)size * n2)};
        auto slice_rsrc = [&](int stage) {
            if constexpr (!REBASE) return group_rs;
            const bool live = stage < nk;
            const int srows = live ? min(BR, size - stage * BR) : 0;
            const size_t row0 = (size_t)row_base + (size_t)(live ? stage * BR : 0);
            return SliceRsrc{make_rsrc_v(p.lhs + row0 * p.k, (uint32_t)srows * k1), make_rsrc_v(p.lhs_scale + row0 * ks, (uint32_t)srows * ks),
                             make_rsrc_v(p.dout + row0 * p.n, (uint32_t)srows * n2)};
        };
        // ring load d of row slice `stage`: 0, 1 codes, 2 scales, 3 .. 6 dout.  FULL: the slice lies inside the group and
        // the column checks are left out: columns past k or n then read the next row's values (or zeros past the
        // descriptor), which only reach output rows or columns that are never stored.
        auto dma_one = [&](auto d_c, int stage, const SliceRsrc& r, auto full_c) {
            constexpr int d = decltype(d_c)::value;
            constexpr bool FULL = decltype(full_c)::value;
            const int slot = stage % STAGES;
            const bool live = stage < nk;
            // (the slice offset goes through readfirstlane, opaque to loop strength reduction: ragged_k_bf16.hip)
            const uint32_t srow = (uint32_t)(REBASE ? 0 : __builtin_amdgcn_readfirstlane(stage * BR));
            if constexpr (d < 2) {
                const bool ok = live && 16 * (l & 15) < p.k - i0;
                load_lds16(r.a, lds_c + (uint32_t)slot * SLICE + d * 1024u,
                           FULL || ok ? a_lane + (srow + (uint32_t)(8 * wave_u + 4 * d)) * k1 + (uint32_t)i0 : kOOB);
            } else if constexpr (d == 2) {
                const bool ok = live && 32 * (l & 7) < p.k - i0;
                load_lds1(r.s, lds_s + (uint32_t)slot * 1024u,
                          FULL || ok ? s_lane + (srow + (uint32_t)(8 * wave_u)) * ks + ((uint32_t)i0 >> 5) : kOOB);
            } else {
                constexpr int u = d - 3;
                const bool ok = live && ch8[u] < p.n - j0;
                load_lds16(r.b, lds_b + (uint32_t)slot * (SLICE * 2) + u * 1024u,
                           FULL || ok ? b_lane[u] + (srow + (uint32_t)(2 * (4 * wave_u + u))) * n2 + (uint32_t)j0 * 2u : kOOB);
            }
        };
        // step O of turning slice `stage`, whose codes are in LDS, to bf16 in slot stage % 2
        auto turn_one = [&](auto o_c, Turn& q, int stage) {
            constexpr int O = decltype(o_c)::value;
            const int slot = stage % STAGES;
            if constexpr (O == 0) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    q.c[u] = *(const i32x4*)(&sm.ring.codes[slot][0] + wave * 2048 + u * 1024 + 16 * l);
                    q.byte[u] = sm.ring.scale[slot][wave][8 * (4 * u + (l >> 4)) + ((l & 15) >> 1)];
                }
            }
            if constexpr (O >= 4 && O < 12) {   // two values a conversion, four values a step
                constexpr int w = O - 4, u = w >> 2, d = w & 3;
                const float s = __uint_as_float(q.byte[u] << 23);   // exponent field 255 is NaN to the conversion
                const uint32_t c = (uint32_t)q.c[u][d];
                q.v[2 * u + (d >> 1)][2 * (d & 1)] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false));
                q.v[2 * u + (d >> 1)][2 * (d & 1) + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true));
            }
            if constexpr (O >= 12 && O < 16) {
                constexpr int x = O - 12, u = x >> 1, hf = x & 1;
                *(i32x4*)(&sm.ring.a[stage & 1][0] + off(8 * wave + 4 * u + (l >> 4), 16 * (l & 15) + 8 * hf)) = q.v[x];
            }
        };

        f32x16 acc[MI][NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

        // one half slice: MFMAs on `cur`, each followed by at most one ring load, one fragment read of `nxt` (step s of slot
        // a / b) and, in the first half of an iteration, one step of turning slice `turned`, in a pinned order
        auto phase = [&](auto nb_c, auto half_c, Frags& cur, Frags& nxt, const uint16_t* a, const uint16_t* b, int s,
                         int stage, int turned, auto full_c) {
            constexpr int NB = decltype(nb_c)::value;
            constexpr int HALF = decltype(half_c)::value;   // ring loads: 0 none, 1 the first ones, 2 the rest, with the turning
            constexpr int NM = NB * NJ, NR = NB > 0 ? NB + NJ : 0, ND = HALF == 1 ? FIRST : HALF == 2 ? SECOND : 0;
            constexpr int SP = ND > 0 && NM >= ND ? NM / (ND > 0 ? ND : 1) : 1;   // MFMAs between two ring loads
            constexpr int LD = ND > 0 ? (ND - 1) * SP + 1 : 0, NC = HALF == 2 ? 16 : 0;
            constexpr int N1 = NM > NR ? (NM > LD ? NM : LD) : (NR > LD ? NR : LD), NOPS = N1 > NC ? N1 : NC;
            const SliceRsrc rs = slice_rsrc(stage);
            Turn q;
            static_for<0, NOPS>([&](auto o_c) {
                constexpr int o = decltype(o_c)::value;
                if constexpr (o < NM) {
                    constexpr int i = o % (NB > 0 ? NB : 1), j = o / (NB > 0 ? NB : 1);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cur.b[j], cur.a[i], acc[i][j], 0, 0, 0);
                }
                if constexpr (ND > 0 && o % SP == 0 && o / SP < ND)
                    dma_one(std::integral_constant<int, (HALF - 1) * FIRST + o / SP>{}, stage, rs, full_c);
                if constexpr (HALF == 2) turn_one(o_c, q, turned);
                if constexpr (o < NR) read_one<NB, o>(nxt, a, b, s, r0w, c0w);
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        auto run = [&](auto nb_c) {
            constexpr int NB = decltype(nb_c)::value;
            Frags f0, f1;
            // Slice s's first loads go out in the second half of iteration s - 4 (its code slot was turned in iteration
            // s - 5, its dout slot is free once the barrier of iteration s - 4 has passed), the rest in the first half of
            // iteration s - 3.  Iteration kt turns slice kt + 1 before its barrier: 15 loads follow that slice's scales then
            // (one of dout, SECOND, PER, FIRST), and PER * (STAGES - 2) its last one at the barrier.
            static_for<0, STAGES - 1>([&](auto st_c) {
                const SliceRsrc rs = slice_rsrc(decltype(st_c)::value);
                static_for<0, PER>([&](auto d_c) { dma_one(d_c, decltype(st_c)::value, rs, std::false_type{}); });
            });
            const SliceRsrc rs3 = slice_rsrc(STAGES - 1);
            static_for<0, FIRST>([&](auto d_c) { dma_one(d_c, STAGES - 1, rs3, std::false_type{}); });
            wait_vm<PER * (STAGES - 2) + FIRST>();   // slice 0 in LDS
            Turn q;
            static_for<0, 16>([&](auto o_c) { turn_one(o_c, q, 0); });
            lds_barrier();
            if constexpr (NB > 0) static_for<0, NB + NJ>([&](auto r_c) { read_one<NB, decltype(r_c)::value>(f0, sm.ring.a[0], sm.ring.b[0], 0, r0w, c0w); });
            __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): exact wait counts at the loop head
            auto iter = [&](int kt, auto full_c) {
                const int slot = kt % STAGES, ns = (kt + 1) % STAGES;
                wait_vm<1 + SECOND + PER + FIRST>();   // this wave's codes and scales of slice kt + 1 in LDS
                phase(nb_c, std::integral_constant<int, 2>{}, f0, f1, sm.ring.a[kt & 1], sm.ring.b[slot], 1, kt + STAGES - 1, kt + 1, full_c);
                wait_vm<PER * (STAGES - 2)>();   // slice kt + 1 in LDS
                lds_barrier();
                phase(nb_c, std::integral_constant<int, 1>{}, f1, f0, sm.ring.a[(kt + 1) & 1], sm.ring.b[ns], 0, kt + STAGES, 0, full_c);
            };
            // Iterations whose ring loads all fall inside the group skip the range checks and run unrolled by four, the ring's
            // slot count, so that slots are constants; the last ones, up to six, take them at run time and keep the checks.
            auto iter_c = [&](auto r_c, int kt) {
                constexpr int R = decltype(r_c)::value, slot = R % STAGES, ns = (R + 1) % STAGES;
                wait_vm<1 + SECOND + PER + FIRST>();
                phase(nb_c, std::integral_constant<int, 2>{}, f0, f1, sm.ring.a[R & 1], sm.ring.b[slot], 1, kt + STAGES - 1, kt + 1, std::true_type{});
                wait_vm<PER * (STAGES - 2)>();
                lds_barrier();
                phase(nb_c, std::integral_constant<int, 1>{}, f1, f0, sm.ring.a[(R + 1) & 1], sm.ring.b[ns], 0, kt + STAGES, 0, std::true_type{});
            };
            int kt = 0;
            for (; kt + 3 + STAGES < nk; kt += 4) static_for<0, 4>([&](auto r_c) { iter_c(r_c, kt + decltype(r_c)::value); });
            for (; kt + 1 < nk; ++kt) iter(kt, std::false_type{});
            const int last = nk - 1;
            phase(nb_c, std::integral_constant<int, 0>{}, f0, f1, sm.ring.a[last & 1], sm.ring.b[last % STAGES], 1, 0, 0, std::false_type{});
            static_for<0, NB * NJ>([&](auto o_c) {   // the last half slice's MFMAs
                constexpr int o = decltype(o_c)::value, i = o % (NB > 0 ? NB : 1), j = o / (NB > 0 ? NB : 1);
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f1.b[j], f1.a[i], acc[i][j], 0, 0, 0);
            });
        };
        if (nk > 0) with_nb<MI>(nb, run);
        // Every ring load has landed (the zero-fill loads of slices past the end may still be in flight, and the epilogue
        // strips overlap their slots) and every wave is done reading the ring before it is reused.
        wait_vm<0>();
        lds_barrier();

        const rsrc_t ro = make_rsrc((const char*)p.out + (((size_t)grp * p.splits + part) * p.k + i0) * p.n * osz, (uint32_t)(rows_valid * p.n * osz));
        static_assert(4 * 32 * (WCOLS + 4) * 4 <= (int)sizeof(sm.ring), "epilogue strips fit the ring");
        const EpiTile ep{nullptr, p.alpha, p.beta};
        store_acc<MI, NJ, WCOLS, OutT, EPI, true>(acc, reinterpret_cast<float*>(&sm.ring) + wave * 32 * (WCOLS + 4), ro, p.n, j0,
                                                  r0w, c0w, ep);
        lds_barrier();   // strips read before the next tile's ring loads land there
    }
    wait_vm<0>();   // no ring load may still be writing LDS when the workgroup ends
}

// 32-bit buffer offsets over one 32-row slice of lhs / dout and one 256-row output tile
bool ok(const KmxParams& p) {
    const uint64_t a = 33ull * (uint64_t)p.k, b = 33ull * (uint64_t)p.n * 2u, o = 256ull * (uint64_t)p.n * 4u;
    return p.n % 8 == 0 && a < (1ull << 31) && b < (1ull << 31) && o < (1ull << 31) && (uintptr_t)p.lhs % 16 == 0 &&
           (uintptr_t)p.dout % 16 == 0 && (uintptr_t)p.out % 16 == 0;
}
template <bool REBASE>
void launch(const KmxParams& p, int grid, hipStream_t s) {
    const bool epi = p.alpha != 1.f || p.beta != 0.f;
    if (epi) {
        if (p.out_f32) hipLaunchKernelGGL((kernel<true, float, REBASE>), dim3(grid), dim3(NT), 0, s, p);
        else hipLaunchKernelGGL((kernel<true, uint16_t, REBASE>), dim3(grid), dim3(NT), 0, s, p);
    } else {
        if (p.out_f32) hipLaunchKernelGGL((kernel<false, float, REBASE>), dim3(grid), dim3(NT), 0, s, p);
        else hipLaunchKernelGGL((kernel<false, uint16_t, REBASE>), dim3(grid), dim3(NT), 0, s, p);
    }
}

}  // namespace kmxr

template <int MI, int BR, int SLOTS>
static void launch_kmx(const KmxParams& p, int per_cu, int cus, hipStream_t s) {
    const int64_t tiles = (int64_t)p.g * p.splits * ((p.k + 64 * MI - 1) / (64 * MI)) * ((p.n + 255) / 256);
    const dim3 grid((uint32_t)std::max<int64_t>(1, std::min<int64_t>(tiles, (int64_t)per_cu * cus)));
    if (p.out_f32) hipLaunchKernelGGL((kmx::kernel<float, MI, BR, SLOTS>), grid, dim3(kmx::NT), 0, s, p);
    else hipLaunchKernelGGL((kmx::kernel<uint16_t, MI, BR, SLOTS>), grid, dim3(kmx::NT), 0, s, p);
}

// Parts of a group's rows: where the tiles leave half the chip idle, as many as fill it, of at least 256 rows on average
// (13232 rows of one group, k 192, n 4480, 18 tiles: 303 us in one part, 41 + 10 with 14, the 10 for their sum).
int ragged_k_mx_splits(int64_t m, int64_t k, int64_t n, int g) {
    const int64_t tiles = g * ((k + 255) / 256) * ((n + 255) / 256);
    if (tiles == 0 || tiles >= 128) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(32, 256 / tiles), m / (256 * (int64_t)g)));
}

static hipError_t launch_tiles(const KmxParams& p, int cus, hipStream_t s) {
    if (kmxr::ok(p)) {
        const int64_t tiles = (int64_t)p.g * p.splits * ((p.k + 255) / 256) * ((p.n + 255) / 256);
        const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, cus));
        const uint64_t a = ((uint64_t)p.m + 64u) * (uint64_t)p.k, b = ((uint64_t)p.m + 64u) * (uint64_t)p.n * 2u;
        if (a < (1ull << 31) && b < (1ull << 31)) kmxr::launch<false>(p, grid, s);
        else kmxr::launch<true>(p, grid, s);
    } else if ((int64_t)p.m < 64 * (int64_t)p.g) {
        // few rows a group: the output is most of the work, and two workgroups a compute unit overlap one's stores with the
        // other's loads
        launch_kmx<2, 32, 1>(p, 2, cus, s);
    } else {
        launch_kmx<4, 64, 2>(p, 1, cus, s);
    }
    return hipGetLastError();
}

hipError_t launch_ragged_k_mx(const KmxParams& p, int cus, hipStream_t s) {
    if (p.splits == 1) return launch_tiles(p, cus, s);
    KmxParams q = p;
    q.out = q.parts; q.out_f32 = 1; q.alpha = 1.f; q.beta = 0.f;
    const hipError_t e = launch_tiles(q, cus, s);
    if (e != hipSuccess) return e;
    const int64_t per = (int64_t)p.k * p.n;
    const bool four = per % 4 == 0;
    const dim3 grid((uint32_t)((per + (four ? 1024 : 256) - 1) / (four ? 1024 : 256)), p.g);
    if (p.out_f32) {
        if (four) hipLaunchKernelGGL((kmx::add_up<float, 4>), grid, dim3(256), 0, s, p.parts, (float*)p.out, per, p.splits, p.alpha, p.beta);
        else hipLaunchKernelGGL((kmx::add_up<float, 1>), grid, dim3(256), 0, s, p.parts, (float*)p.out, per, p.splits, p.alpha, p.beta);
    } else {
        if (four) hipLaunchKernelGGL((kmx::add_up<uint16_t, 4>), grid, dim3(256), 0, s, p.parts, (uint16_t*)p.out, per, p.splits, p.alpha, p.beta);
        else hipLaunchKernelGGL((kmx::add_up<uint16_t, 1>), grid, dim3(256), 0, s, p.parts, (uint16_t*)p.out, per, p.splits, p.alpha, p.beta);
    }
    return hipGetLastError();
}

}  // namespace gg
