// unpermute_grad.hip -- the gradients of moe_unpermute, out[t] = sum_j w[t, j] y[p(t, j)]:
//   dy[p(t, j)] = w[t, j] dout[t],   dw[t, j] = dout[t] . y[p(t, j)].
// One pass: the waves of token t read its dout row once, and for each of its copies read the copy's y row
// and write its dy row, so every row of dout, y and dy moves once (3 row widths a copy at top_k = 1, tending
// to 2): bound by memory.  dw's partial sums stay in fp32 registers, are added over the wave's lanes by
// exchanges and over the token's waves in LDS, in a fixed order.  4096 tokens of 7168 bf16 columns at
// top_k = 1 / 2 / 8: 38 / 59 / 201 us (4.7 to 5.0 TB/s); 2048 of 7165 at top_k = 6 92 us.  Batches of eight
// for every top_k took 53 / 67 us, element accesses for widths that 16 bytes do not divide 234, and two waves
// for widths of which one wave takes all 126 against 69 us (65536 tokens of 512).
//
// A dy row is written by the one copy that sorted_to_copy names for it (and that points back to it), so the
// result does not depend on the order of waves even for index arrays that no permute wrote; rows that no
// copy claims are found and cleared by the workgroups behind the tokens'.
#include "common.hpp"
#include "launch.hpp"
#include "ring.hpp"

namespace gg {
namespace upg {

constexpr int KB = 8;       // copies handled at a time
constexpr int CLEAR = 16;   // rows that a clearing wave looks over at a time (64: 22 us, not 12, where 46 of 183 rows of 1030 are lost)

__device__ inline float up(uint32_t u) { return __uint_as_float(u); }

// eight consecutive elements as floats; rows begin where the width puts them, so the 16-byte accesses are
// aligned to an element only (the target's global memory takes that)
typedef i32x4 __attribute__((aligned(2))) i32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
__device__ inline void load8(const uint16_t* p, float (&v)[8]) {
    const i32x4 q = __builtin_nontemporal_load((const i32x4_any*)p);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = up((uint32_t)q[e] << 16);
        v[2 * e + 1] = up((uint32_t)q[e] & 0xffff0000u);
    }
}
__device__ inline void load8(const float* p, float (&v)[8]) {
    const f32x4 a = __builtin_nontemporal_load((const f32x4_any*)p), b = __builtin_nontemporal_load((const f32x4_any*)(p + 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
    }
}
__device__ inline void store8(uint16_t* p, const float (&v)[8]) {
    const i32x4 q = {(int)ring::pack_bf16(v[0], v[1]), (int)ring::pack_bf16(v[2], v[3]), (int)ring::pack_bf16(v[4], v[5]),
                     (int)ring::pack_bf16(v[6], v[7])};
    __builtin_nontemporal_store(q, (i32x4_any*)p);
}
__device__ inline void store8(float* p, const float (&v)[8]) {
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4_any*)p);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4_any*)(p + 4));
}
__device__ inline float ld1(const uint16_t* p) { return up((uint32_t)*p << 16); }
__device__ inline float ld1(const float* p) { return *p; }
__device__ inline void st1(uint16_t* p, float v) { *p = f32_to_bf16(v); }
__device__ inline void st1(float* p, float v) { *p = v; }

// WPT waves share a token (4 / WPT tokens a workgroup)
template <typename T, bool VEC, int WPT>
__global__ __launch_bounds__(256) void kernel(UnpermuteGradArgs a, int tok_blocks) {
    __shared__ float part[4][KB];
    const int l = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int M = a.tokens * a.top_k, n = a.n;
    T* dy = (T*)a.dy;
    if ((int)blockIdx.x >= tok_blocks) {   // clear the rows that no copy claims
        const int nw = ((int)gridDim.x - tok_blocks) * 4;
        for (int64_t p0 = (int64_t)(((int)blockIdx.x - tok_blocks) * 4 + wv) * CLEAR; p0 < M; p0 += (int64_t)nw * CLEAR) {
            const int64_t p = p0 + l;
            bool lost = false;
            if (l < CLEAR && p < M) {
                const int i = a.sorted_to_copy[p];
                lost = i < 0 || i >= M || a.copy_to_sorted[i] != p;
            }
            for (uint64_t rows = __ballot(lost); rows; rows &= rows - 1) {
                T* o = dy + (size_t)(p0 + __ffsll((unsigned long long)rows) - 1) * n;
                if constexpr (VEC) {
                    const float zero[8] = {};
                    for (uint32_t c = 8 * l; c < (uint32_t)n; c += 512) store8(o + min((int)c, n - 8), zero);
                } else {
                    for (int c = l; c < n; c += 64) st1(o + c, 0.f);
                }
            }
        }
        return;
    }
    const int t = blockIdx.x * (4 / WPT) + wv / WPT, h = wv % WPT;
    const bool on = t < a.tokens;
    const T* drow = (const T*)a.dout + (size_t)(on ? t : 0) * n;
    for (int j0 = 0; j0 < a.top_k; j0 += KB) {
        float acc[KB], w[KB];
        int pos[KB];
        bool claim[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            acc[j] = 0.f;
            pos[j] = -1;
            w[j] = 0.f;
            claim[j] = false;
            if (on && j0 + j < a.top_k) {
                const int i = t * a.top_k + j0 + j, p = a.copy_to_sorted[i];
                w[j] = a.weights[i];
                if (p >= 0 && p < M) {
                    pos[j] = p;
                    claim[j] = a.sorted_to_copy[p] == i;
                }
            }
        }
        if (on) {
            if constexpr (VEC) {
                // (a row's last eight elements may overlap the eight before: their dy is written twice, the same,
                // and their products are left out of the second sum)
                auto columns = [&](auto k_c) {
                    constexpr int K = decltype(k_c)::value;   // copies whose rows are read: absent ones among them read row 0
                    for (uint32_t c0 = 512 * h + 8 * l; c0 < (uint32_t)n; c0 += 512 * WPT) {   // (may pass 2^31)
                        const int c = min((int)c0, n - 8), done = (int)c0 - c;
                        float d[8];
                        load8(drow + c, d);
                        float y[K][8];
#pragma unroll
                        for (int j = 0; j < K; ++j) load8((const T*)a.y + (size_t)(pos[j] < 0 ? 0 : pos[j]) * n + c, y[j]);
#pragma unroll
                        for (int j = 0; j < K; ++j) {
                            float o[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                acc[j] = __builtin_fmaf(e < done ? 0.f : d[e], pos[j] < 0 || e < done ? 0.f : y[j][e], acc[j]);
                                o[e] = w[j] * d[e];
                            }
                            if (claim[j]) store8(dy + (size_t)pos[j] * n + c, o);
                        }
                    }
                };
                // (loads behind a branch each would wait for one another; a batch of eight where there are two
                // copies costs half the speed)
                if (a.top_k - j0 > 4) columns(std::integral_constant<int, 8>{});
                else if (a.top_k - j0 > 2) columns(std::integral_constant<int, 4>{});
                else if (a.top_k - j0 > 1) columns(std::integral_constant<int, 2>{});
                else columns(std::integral_constant<int, 1>{});
            } else {
                for (int c = 64 * h + l; c < n; c += 64 * WPT) {
                    const float d = ld1(drow + c);
#pragma unroll
                    for (int j = 0; j < KB; ++j) {
                        if (pos[j] < 0) continue;
                        acc[j] = __builtin_fmaf(d, ld1((const T*)a.y + (size_t)pos[j] * n + c), acc[j]);
                        if (claim[j]) st1(dy + (size_t)pos[j] * n + c, w[j] * d);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (pos[j] < 0) acc[j] = 0.f;   // (its terms were dout times 0, and dout need not be finite)
#pragma unroll
            for (int s = 32; s > 0; s >>= 1) acc[j] += __shfl_xor(acc[j], s, 64);
        }
        if constexpr (WPT > 1) {
            __syncthreads();
            if (l == 0)
#pragma unroll
                for (int j = 0; j < KB; ++j) part[wv][j] = acc[j];
            __syncthreads();
            if (on && h == 0 && l < KB && j0 + l < a.top_k) {
                float v = part[wv][l];
#pragma unroll
                for (int q = 1; q < WPT; ++q) v += part[wv + q][l];
                a.dweights[(size_t)t * a.top_k + j0 + l] = v;
            }
        } else {
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (on && l == j && j0 + j < a.top_k) a.dweights[(size_t)t * a.top_k + j0 + j] = acc[j];
        }
    }
}

template <typename T, int WPT>
hipError_t launch_w(const UnpermuteGradArgs& a, hipStream_t s) {
    const int tpb = 4 / WPT, tok_blocks = (int)(((int64_t)a.tokens + tpb - 1) / tpb);
    const int64_t M = (int64_t)a.tokens * a.top_k;
    const int clear = (int)((M + 4 * CLEAR - 1) / (4 * CLEAR) < 512 ? (M + 4 * CLEAR - 1) / (4 * CLEAR) : 512);
    if ((int64_t)tok_blocks + clear > kMaxBlocks) return hipErrorInvalidConfiguration;
    if (a.n >= 8) hipLaunchKernelGGL((kernel<T, true, WPT>), dim3(tok_blocks + clear), dim3(256), 0, s, a, tok_blocks);
    else hipLaunchKernelGGL((kernel<T, false, WPT>), dim3(tok_blocks + clear), dim3(256), 0, s, a, tok_blocks);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const UnpermuteGradArgs& a, hipStream_t s) {
    return a.n <= 512 ? launch_w<T, 1>(a, s) : launch_w<T, 2>(a, s);   // (a second wave would have no columns)
}

}  // namespace upg

hipError_t launch_unpermute_grad(const UnpermuteGradArgs& a, bool bf16, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    return bf16 ? upg::launch_t<uint16_t>(a, s) : upg::launch_t<float>(a, s);
}

}  // namespace gg
