// lora.hip -- low-rank adapters of many requests (or experts) at once, beside a shared projection, and their
// gradients on gfx950.  Row i of x has adapter h (its group of sorted rows, or row_group[i]), or none:
//   v[i] = x[i] . a[h]^T,   out[i] = base[i] + s[h] v[i] . b[h]^T          a [g, r, k], b [g, n, r]
//   u[i] = dout[i] . b[h],  dx[i] = dbase[i] + s[h] u[i] . a[h],
//   da[h] = s[h] sum_i u[i]^T x[i],  db[h] = s[h] sum_i dout[i]^T v[i].
// r is small beside k and n, so all of it is bound by reading x, base and dout and writing out and dx once.
//
// Three kernels.  `shrink` contracts the long axis (v, u): a tile of rows of one adapter against its r rows of
// weights, the axis split over the four waves of a workgroup and, for few rows, over workgroups.  `expand` contracts
// r and adds the other term.  `outer` contracts the rows of a group (da, db), in chunks of rows that `join` adds up
// in order where a group has more than one: no atomics, so results do not depend on the launch.
// The backward pass is the forward one with the weights' axes swapped, so `turn` writes b as [g, r, n] and a as
// [g, k, r] once a call, which is small, and `shrink` and `expand` serve both.
//
// Products of bf16 weights with the fp32 v and u run on the bf16 matrix instructions with v and u as a sum of two
// bf16 values (16 bits of fraction, so their error stays below a bf16 result's and 2^-17 of an fp32 one), of three
// (24 bits) in the row sums that leave in fp32.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace gg {
namespace lora {

constexpr int NT = 256;
constexpr int KC = 64;           // elements of the long axis that a wave takes at a time
constexpr int MAXCHUNK = 2048;   // rows in any order: of these many, a workgroup takes those of its adapter

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// 16 bytes that may begin at any element (the target's global memory takes that)
typedef i32x4 __attribute__((aligned(2))) i32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

// Eight consecutive elements of a contracted axis, as the matrix instructions take them from one lane: lanes
// 16 q .. 16 q + 15 hold elements 8 q .. 8 q + 7 of 32.  fp32 runs as eight instructions of four elements, where
// instruction i takes element 8 q + i of group q.
template <typename T> struct Frag;
template <> struct Frag<uint16_t> {
    bf16x8 v;
    __device__ void load(const uint16_t* p) { v = __builtin_bit_cast(bf16x8, (i32x4)*(const i32x4_any*)p); }
    __device__ void load_lds(const uint16_t* p) { v = *(const bf16x8*)p; }
    __device__ void load_part(const uint16_t* p, int valid) {   // elements past `valid` are 0
        i32x4 q = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) q[e >> 1] |= (int)((uint32_t)p[e] << (16 * (e & 1)));
        v = __builtin_bit_cast(bf16x8, q);
    }
    __device__ static f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
    }
};
template <> struct Frag<float> {
    f32x4 lo, hi;
    __device__ void load(const float* p) { lo = *(const f32x4_any*)p; hi = *(const f32x4_any*)(p + 4); }
    __device__ void load_lds(const float* p) { lo = *(const f32x4*)p; hi = *(const f32x4*)(p + 4); }
    __device__ void load_part(const float* p, int valid) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo[e] = e < valid ? p[e] : 0.f;
            hi[e] = e + 4 < valid ? p[e + 4] : 0.f;
        }
    }
    __device__ static f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[e], b.lo[e], c, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi[e], b.hi[e], c, 0, 0, 0);
        return c;
    }
};

// P bf16 values that add up to x: each holds what the ones before it left.  An infinity or a NaN stays in the first.
template <int P>
__device__ inline void split(float x, uint16_t (&out)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const __bf16 b = (__bf16)x;
        out[i] = __builtin_bit_cast(uint16_t, b);
        const float left = x - (float)b;
        x = __builtin_isfinite(left) ? left : 0.f;
    }
}

// Which rows a workgroup has: `rows` of adapter h (-1: rows without one), row i being first + i or list[i].
struct RowTile { int h, rows, first; const int* list; };
struct RowSmem {
    union {
        Tables tab;
        struct { int list[MAXCHUNK]; int wave[4]; } any;
    };
};

// Sorted rows: tile `id` of `tm` rows each, adapters first and then the rows behind the last one's.
__device__ inline RowTile sorted_tile(const Rows& p, int id, int tm, RowSmem& sm) {
    int tiles, covered;
    build_tables<NT>(p.group_sizes, p.g, p.m, tm, 1, sm.tab, &tiles, &covered);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && p.status) *p.status = sm.tab.flags;
    if (id < tiles) {
        const int h = find_group(sm.tab.tile_off, p.g, id);
        const int first = sm.tab.row_off[h] + (id - sm.tab.tile_off[h]) * tm;
        return {h, min(tm, sm.tab.row_off[h + 1] - first), first, nullptr};
    }
    const int first = covered + (id - tiles) * tm;
    return {-1, max(0, min(tm, p.m - first)), first, nullptr};
}
// Rows in any order: slot `id` of a chunk is adapter `id`, or (fewer rows than adapters) the adapter of row `id` of
// the chunk if no row before it has the same; the last slot is the rows without one.  The list is in row order.
__device__ inline RowTile any_tile(const Rows& p, int id, RowSmem& sm) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && p.status) *p.status = 0;
    const int slots = p.slots + 1, c = id / slots, slot = id - c * slots;
    const int r0 = c * p.chunk, n = min(p.chunk, p.m - r0);
    const bool by_row = p.slots < p.g;
    int h = slot;
    if (slot == p.slots) h = -1;
    else if (by_row) {
        if (slot >= n) return {-1, 0, 0, nullptr};
        h = p.row_group[r0 + slot];
        if (h < 0 || h >= p.g) return {-1, 0, 0, nullptr};
    }
    const int t = threadIdx.x, w = t >> 6;
    int found = 0;
    for (int i0 = 0; i0 < n; i0 += NT) {
        const int i = i0 + t;
        int of = i < n ? p.row_group[r0 + i] : INT32_MIN;
        if (i < n && (of < 0 || of >= p.g)) of = -1;
        const unsigned long long mine = __ballot(of == h);
        if ((t & 63) == 0) sm.any.wave[w] = __popcll(mine);
        __syncthreads();
        int at = found;
        for (int j = 0; j < 4; ++j) {
            if (j < w) at += sm.any.wave[j];
            found += sm.any.wave[j];
        }
        if (of == h) sm.any.list[at + __popcll(mine & ((1ull << (t & 63)) - 1))] = r0 + i;
        __syncthreads();
    }
    if (by_row && h >= 0 && found > 0 && sm.any.list[0] != r0 + slot) found = 0;   // an earlier row's slot has them
    return {h, found, 0, sm.any.list};
}
__device__ inline RowTile row_tile(const Rows& p, int id, int tm, RowSmem& sm) {
    return p.group_sizes ? sorted_tile(p, id, tm, sm) : any_tile(p, id, sm);
}
__device__ inline int row_at(const RowTile& w, int i) { return w.list ? w.list[i] : w.first + i; }

// ---------------------------------------------------------------------------------------------------------------
// shrink: t[split, row, j] = x[row] . w[h][j], over the split's part of the long axis.  16 MT rows, 16 NB columns j.
// The weights are the first operand, so a lane ends with four consecutive j of one row.

template <typename T, int NB, int MT>
__global__ __launch_bounds__(NT) void shrink(Shrink p) {
    constexpr int TM = 16 * MT;
    __shared__ RowSmem rs;
    __shared__ f32x4 red[2][MT * NB * 64];
    const RowTile w = row_tile(p.rows, blockIdx.x, TM, rs);
    if (w.h < 0 || w.rows == 0) return;
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;
    const int nch = (p.k + KC - 1) / KC, per = (nch + (int)gridDim.y - 1) / (int)gridDim.y;
    const int c0 = blockIdx.y * per, c1 = min(nch, c0 + per);
    const T* wp[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wp[b] = (const T*)p.w + ((int64_t)w.h * p.r + min(16 * b + i16, p.r - 1)) * p.k + 8 * q;
    for (int r0 = 0; r0 < w.rows; r0 += TM) {
        const T* xp[MT];
#pragma unroll
        for (int a = 0; a < MT; ++a) xp[a] = (const T*)p.x + (int64_t)row_at(w, min(r0 + 16 * a + i16, w.rows - 1)) * p.stride + 8 * q;
        f32x4 acc[MT][NB];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int whole = min(c1, p.k / KC);   // chunks that lie inside the axis
        for (int c = c0 + wave; c < whole; c += 4) {
            Frag<T> x[MT][2], m[NB][2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int a = 0; a < MT; ++a) x[a][s].load(xp[a] + (int64_t)c * KC + 32 * s);
#pragma unroll
                for (int b = 0; b < NB; ++b) m[b][s].load(wp[b] + (int64_t)c * KC + 32 * s);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int a = 0; a < MT; ++a) acc[a][b] = Frag<T>::mma(m[b][s], x[a][s], acc[a][b]);
        }
        if (c0 <= whole && whole < c1 && (whole - c0) % 4 == wave) {   // the chunk that the axis ends in
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int valid = p.k - whole * KC - 32 * s - 8 * q;
                Frag<T> x[MT], m[NB];
#pragma unroll
                for (int a = 0; a < MT; ++a) x[a].load_part(xp[a] + (int64_t)whole * KC + 32 * s, valid);
#pragma unroll
                for (int b = 0; b < NB; ++b) m[b].load_part(wp[b] + (int64_t)whole * KC + 32 * s, valid);
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int a = 0; a < MT; ++a) acc[a][b] = Frag<T>::mma(m[b], x[a], acc[a][b]);
            }
        }
        // waves 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
        for (int half = 2; half >= 1; half >>= 1) {
            if (wave >= half && wave < 2 * half)
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < NB; ++b) red[wave - half][(a * NB + b) * 64 + l] = acc[a][b];
            __syncthreads();
            if (wave < half)
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[a][b] += red[wave][(a * NB + b) * 64 + l];
            __syncthreads();
        }
        if (wave == 0) {
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                if (r0 + 16 * a + i16 >= w.rows) continue;
                float* to = p.t + ((int64_t)blockIdx.y * p.rows.m + row_at(w, r0 + 16 * a + i16)) * p.r;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 16 * b + 4 * q + e;
                        if (j < p.r) to[j] = acc[a][b][e];
                    }
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------------------
// expand: out[row] = base[row] + s[h] t[row] . w[h]^T for 16 MT rows and `cols` columns, t being the sum of the
// splits.  The weights are the first operand; row i of two 16-row blocks j = 0, 1 is column 8 (i / 4) + 4 j + i % 4 of
// 32, so a lane ends with eight consecutive columns of one row.

template <typename O> struct Out8;
template <> struct Out8<uint16_t> {
    i32x4 q;
    __device__ void load(const uint16_t* p) { q = __builtin_nontemporal_load((const i32x4_any*)p); }
    __device__ float get(int i) const { return __uint_as_float((i & 1) ? (uint32_t)q[i >> 1] & 0xffff0000u : (uint32_t)q[i >> 1] << 16); }
    __device__ void zero() { q = i32x4{0, 0, 0, 0}; }
    __device__ static float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
    __device__ static void put(uint16_t* p, float v) { const __bf16 b = (__bf16)v; *p = __builtin_bit_cast(uint16_t, b); }
    __device__ static void store(uint16_t* p, const float (&v)[8]) {
        i32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
            w[i] = __builtin_bit_cast(int, b);
        }
        __builtin_nontemporal_store(w, (i32x4_any*)p);
    }
};
template <> struct Out8<float> {
    f32x4 a, b;
    __device__ void load(const float* p) {
        a = __builtin_nontemporal_load((const f32x4_any*)p);
        b = __builtin_nontemporal_load((const f32x4_any*)(p + 4));
    }
    __device__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
    __device__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ static float one(const float* p) { return *p; }
    __device__ static void put(float* p, float v) { *p = v; }
    __device__ static void store(float* p, const float (&v)[8]) {
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4_any*)p);
        __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4_any*)(p + 4));
    }
};

// t of a tile's rows as the second operand: `width` elements a row, bf16: [high | low] of 8 ceil(r / 8) each.
template <typename T, int NB> struct Narrow {
    static constexpr bool BF = sizeof(T) == 2;
    static constexpr int PITCH = BF ? 32 * NB + 8 : 16 * (NB < 2 ? 2 : NB) + 4;
};

template <typename T, typename O, int NB, int MT, bool WHOLE>   // WHOLE: r % 8 == 0
__global__ __launch_bounds__(NT) void expand(Expand p) {
    constexpr int TM = 16 * MT, PITCH = Narrow<T, NB>::PITCH;
    constexpr bool BF = sizeof(T) == 2;
    __shared__ RowSmem rs;
    __shared__ __attribute__((aligned(16))) T nar[TM * PITCH];
    const int ct = blockIdx.x % p.col_tiles, id = blockIdx.x / p.col_tiles;
    const RowTile w = row_tile(p.rows, id, TM, rs);
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;
    const int col0 = ct * p.cols, col1 = min(p.n, col0 + p.cols);
    const O* base = (const O*)p.base;
    O* out = (O*)p.out;
    if (w.h < 0) {   // rows without an adapter: what was there
        for (int i = 0; i < w.rows; ++i) {
            const int64_t row = row_at(w, i);
            if (p.v && ct == 0)
                for (int j = t; j < p.r; j += NT) p.v[row * p.r + j] = 0.f;
            if (base == out && p.base_stride == p.out_stride) continue;
            for (int c = col0 + t; c < col1; c += NT) out[row * p.out_stride + c] = base ? base[row * p.base_stride + c] : (O)0;
        }
        return;
    }
    const float scale = p.scaling ? p.scaling[w.h] : 1.f;
    const int rk = (p.r + 7) / 8;                       // eights of r
    const int eights = BF ? 2 * rk : rk, steps = (eights + 3) / 4;
    const T* wb = (const T*)p.w + (int64_t)w.h * p.n * p.r;
    for (int r0 = 0; r0 < w.rows; r0 += TM) {
        if (r0) __syncthreads();
        for (int e = t; e < TM * 8 * rk; e += NT) {
            const int i = e / (8 * rk), j = e - i * 8 * rk;
            float s = 0.f;
            if (r0 + i < w.rows && j < p.r) {
                const int64_t at = (int64_t)row_at(w, r0 + i) * p.r + j;
                for (int k = 0; k < p.splits; ++k) s += p.t[(int64_t)k * p.rows.m * p.r + at];
                if (p.v && ct == 0 && p.v != p.t) p.v[at] = s;
            }
            s *= scale;
            if constexpr (BF) {
                uint16_t two[2];
                split<2>(s, two);
                nar[i * PITCH + j] = two[0];
                nar[i * PITCH + 8 * rk + j] = two[1];
            } else {
                nar[i * PITCH + j] = s;
            }
        }
        for (int e = t; e < TM * 8 * (4 * steps - eights); e += NT) {   // up to whole steps
            const int per = 8 * (4 * steps - eights), i = e / per;
            nar[i * PITCH + 8 * eights + e - i * per] = (T)0;
        }
        __syncthreads();
        for (int c = col0 + 32 * wave; c < col1; c += 128) {
            const int cc = c + 8 * q;   // the lane's eight columns
            Out8<O> o[MT];
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                o[a].zero();
                const int i = r0 + 16 * a + i16;
                if (base && i < w.rows && cc + 8 <= p.n) o[a].load(base + (int64_t)row_at(w, i) * p.base_stride + cc);
            }
            const T* wr[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) wr[j] = wb + (int64_t)min(c + 8 * (i16 >> 2) + 4 * j + (i16 & 3), p.n - 1) * p.r;
            f32x4 acc[MT][2];
#pragma unroll
            for (int a = 0; a < MT; ++a) acc[a][0] = acc[a][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int s = 0; s < steps; ++s) {
                int e = min(4 * s + q, eights - 1);      // past the end: times the zeros above
                if (BF && e >= rk) e -= rk;              // the low parts take the same weights
                Frag<T> m[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (WHOLE) m[j].load(wr[j] + 8 * e);
                    else m[j].load_part(wr[j] + 8 * e, p.r - 8 * e);
                }
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    Frag<T> x;
                    x.load_lds(nar + (16 * a + i16) * PITCH + 8 * (4 * s + q));
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[a][j] = Frag<T>::mma(m[j], x, acc[a][j]);
                }
            }
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                const int i = r0 + 16 * a + i16;
                if (i >= w.rows || cc >= col1) continue;
                const int64_t row = row_at(w, i);
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) { v[e] = acc[a][0][e]; v[4 + e] = acc[a][1][e]; }
                if (cc + 8 <= p.n) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += o[a].get(e);
                    Out8<O>::store(out + row * p.out_stride + cc, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (cc + e < p.n)
                            Out8<O>::put(out + row * p.out_stride + cc + e,
                                         v[e] + (base ? Out8<O>::one(base + row * p.base_stride + cc + e) : 0.f));
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------------------
// turn: [g, rows, cols] -> [g, cols, rows]

template <typename T>
__global__ __launch_bounds__(NT) void turn(const T* __restrict__ a, T* __restrict__ at, int rows, int cols, int tr, int tc) {
    __shared__ T s[32][33];
    const int id = blockIdx.x, c0 = 32 * (id % tc), r0 = 32 * ((id / tc) % tr);
    const int64_t h = id / tc / tr, off = h * rows * cols;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (r0 + y + i < rows && c0 + x < cols) s[y + i][x] = a[off + (int64_t)(r0 + y + i) * cols + c0 + x];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (c0 + y + i < cols && r0 + x < rows) at[off + (int64_t)(c0 + y + i) * rows + r0 + x] = s[x][y + i];
}

// ---------------------------------------------------------------------------------------------------------------
// outer: sums over rows.  A workgroup takes a chunk of rows of one group and TC columns of x (then da [r, k]) or of
// dout (then db [n, r]), 32 rows at a time through LDS; both operands have the rows as their slow axis and are read
// with the transposing LDS reads.  The narrow operand (u or v) is the first, so a lane ends with four consecutive j
// of one column.

enum Wide { BF16 = 0, FP32 = 1, E4M3 = 2 };

// the wide operand's 32 rows in LDS
constexpr int WP16 = 256 + 16, WP32 = 256 + 4;

template <bool F32, int NB, int P> struct OuterSmem;
template <int NB, int P> struct OuterSmem<false, NB, P> {
    __attribute__((aligned(16))) uint16_t wide[2][32 * WP16];
    __attribute__((aligned(16))) uint16_t nar[2][P][32 * (16 * NB + 8)];
};
template <int NB, int P> struct OuterSmem<true, NB, P> {
    __attribute__((aligned(16))) float wide[2][32 * WP32];
    __attribute__((aligned(16))) float nar[2][1][32 * (16 * NB + 4)];
};

// 8 rows (of 32) of one column, from two transposing reads of 4 x 16 values
__device__ inline bf16x8 column8(const uint16_t* base, int pitch, int col0) {
    const int l = threadIdx.x & 63, q = l >> 4, i = l & 15;
    const uint16_t* p = base + (8 * q + (i >> 2)) * pitch + col0 + 4 * (i & 3);
    const i16x4 lo = lds_read_tr16(p), hi = lds_read_tr16(p + 4 * pitch);
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
}

// what a thread holds of the next 32 rows
template <Wide W> struct WideRegs;
template <> struct WideRegs<BF16> {   // row t / 32 + 8 i, eight columns at 8 (t % 32)
    i32x4 v[4];
    __device__ void load(const Outer& p, int row0, int rows, int c0, int cols, int64_t stride, const void* src) {
        const int t = threadIdx.x, c = c0 + 8 * (t & 31);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (t >> 5) + 8 * i;
            v[i] = i32x4{0, 0, 0, 0};
            if (r >= rows || c >= cols) continue;
            const uint16_t* at = (const uint16_t*)src + (int64_t)(row0 + r) * stride + c;
            if (c + 8 <= cols) v[i] = *(const i32x4_any*)at;
            else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < cols) v[i][e >> 1] |= (int)((uint32_t)at[e] << (16 * (e & 1)));
            }
        }
    }
    __device__ void store(uint16_t* to) const {
        const int t = threadIdx.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) *(i32x4*)(to + ((t >> 5) + 8 * i) * WP16 + 8 * (t & 31)) = v[i];
    }
};
template <> struct WideRegs<FP32> {   // row t / 32 + 8 i, eight columns
    f32x4 v[4][2];
    __device__ void load(const Outer& p, int row0, int rows, int c0, int cols, int64_t stride, const void* src) {
        const int t = threadIdx.x, c = c0 + 8 * (t & 31);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (t >> 5) + 8 * i;
            v[i][0] = v[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (r >= rows || c >= cols) continue;
            const float* at = (const float*)src + (int64_t)(row0 + r) * stride + c;
            if (c + 8 <= cols) { v[i][0] = *(const f32x4_any*)at; v[i][1] = *(const f32x4_any*)(at + 4); }
            else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < cols) v[i][e >> 2][e & 3] = at[e];
            }
        }
    }
    __device__ void store(float* to) const {
        const int t = threadIdx.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float* at = to + ((t >> 5) + 8 * i) * WP32 + 8 * (t & 31);
            *(f32x4*)at = v[i][0];
            *(f32x4*)(at + 4) = v[i][1];
        }
    }
};
template <> struct WideRegs<E4M3> {   // row t / 8, one block of 32 columns at 32 (t % 8)
    i32x4 v[2];
    int byte;
    __device__ void load(const Outer& p, int row0, int rows, int c0, int cols, int64_t stride, const void* src) {
        const int t = threadIdx.x, r = t >> 3, c = c0 + 32 * (t & 7);
        v[0] = v[1] = i32x4{0, 0, 0, 0};
        byte = 0;
        if (r < rows && c < cols) {
            const i32x4* at = (const i32x4*)((const uint8_t*)src + (int64_t)(row0 + r) * stride + c);
            v[0] = at[0];
            v[1] = at[1];
            byte = p.x_scale[(int64_t)(row0 + r) * (stride >> 5) + (c >> 5)];
        }
    }
    __device__ void store(uint16_t* to) const {
        const int t = threadIdx.x;
        const float s = __uint_as_float((uint32_t)byte << 23);   // exponent field 255 is NaN to the conversion
        uint16_t* at = to + (t >> 3) * WP16 + 32 * (t & 7);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            i32x4 q;
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const uint32_t c = (uint32_t)v[i >> 1][2 * (i & 1) + d];
                q[2 * d] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false));
                q[2 * d + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true));
            }
            *(i32x4*)(at + 8 * i) = q;
        }
    }
};

template <Wide XW, int NB, int P, int CB>   // XW: x's type; CB: 16-column blocks a wave
__global__ __launch_bounds__(NT) void outer(Outer p) {
    constexpr bool F32 = XW == FP32;
    constexpr int TC = 64 * CB;
    constexpr int NPITCH = 16 * NB + (F32 ? 4 : 8);
    using E = typename std::conditional<F32, float, uint16_t>::type;
    __shared__ Tables tab;
    __shared__ OuterSmem<F32, NB, P> sm;
    static_assert(TC <= 256, "the staged columns");
    int tiles, covered;
    build_tables<NT>(p.group_sizes, p.g, p.m, p.chunk, 1, tab, &tiles, &covered);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = tab.flags;
    const int xt = (p.k + TC - 1) / TC, dt = (p.n + TC - 1) / TC;
    const int id = blockIdx.x / (xt + dt), ct = blockIdx.x - id * (xt + dt);
    if (id >= tiles) return;
    const int h = find_group(tab.tile_off, p.g, id), part = id - tab.tile_off[h];
    const int first = tab.row_off[h] + part * p.chunk, rows = min(p.chunk, tab.row_off[h + 1] - first);
    const bool of_x = ct < xt;
    const int c0 = (of_x ? ct : ct - xt) * TC, cols = of_x ? p.k : p.n;
    const float* nsrc = of_x ? p.u : p.v;
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;

    f32x4 acc[NB][CB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < CB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    constexpr int NPER = 32 * 16 * NB / NT;   // narrow values a thread
    auto body = [&](auto wide_c) {
        constexpr Wide W = decltype(wide_c)::value;
        WideRegs<W> wr;
        float nr[NPER];
        const void* src = of_x ? p.x : p.dout;
        const int64_t stride = of_x ? p.k : p.n;
        auto load = [&](int r0) {
            wr.load(p, first + r0, rows - r0, c0, min(cols, c0 + TC), stride, src);
#pragma unroll
            for (int e = 0; e < NPER; ++e) {
                const int at = t + NT * e, i = at / (16 * NB), j = at % (16 * NB);
                nr[e] = i < rows - r0 && j < p.r ? nsrc[(int64_t)(first + r0 + i) * p.r + j] : 0.f;
            }
        };
        auto store = [&](int slot) {
            wr.store(sm.wide[slot]);
#pragma unroll
            for (int e = 0; e < NPER; ++e) {
                const int at = t + NT * e, i = at / (16 * NB), j = at % (16 * NB);
                if constexpr (F32) sm.nar[slot][0][i * NPITCH + j] = nr[e];
                else {
                    uint16_t s[P];
                    split<P>(nr[e], s);
#pragma unroll
                    for (int z = 0; z < P; ++z) sm.nar[slot][z][i * NPITCH + j] = s[z];
                }
            }
        };
        load(0);
        store(0);
        __syncthreads();
        int slot = 0;
        for (int r0 = 0; r0 < rows; r0 += 32, slot ^= 1) {
            const bool more = r0 + 32 < rows;
            if (more) load(r0 + 32);
            const E* wd = sm.wide[slot];
            if constexpr (F32) {
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    float b[CB];
#pragma unroll
                    for (int c = 0; c < CB; ++c) b[c] = wd[(4 * s + q) * WP32 + 16 * (CB * wave + c) + i16];
#pragma unroll
                    for (int a = 0; a < NB; ++a) {
                        const float n = sm.nar[slot][0][(4 * s + q) * NPITCH + 16 * a + i16];
#pragma unroll
                        for (int c = 0; c < CB; ++c) acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(n, b[c], acc[a][c], 0, 0, 0);
                    }
                }
            } else {
                bf16x8 b[CB];
#pragma unroll
                for (int c = 0; c < CB; ++c) b[c] = column8(wd, WP16, 16 * (CB * wave + c));
#pragma unroll
                for (int a = 0; a < NB; ++a)
#pragma unroll
                    for (int z = 0; z < P; ++z) {
                        const bf16x8 n = column8(sm.nar[slot][z], NPITCH, 16 * a);
#pragma unroll
                        for (int c = 0; c < CB; ++c) acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n, b[c], acc[a][c], 0, 0, 0);
                    }
            }
            if (more) store(slot ^ 1);
            __syncthreads();
        }
    };
    if constexpr (XW == E4M3) {
        if (of_x) body(std::integral_constant<Wide, E4M3>{});
        else body(std::integral_constant<Wide, BF16>{});
    } else {
        body(std::integral_constant<Wide, XW>{});
    }

    // one chunk: the result; more: the chunk's part, at a place that no other chunk of such a group has (two such
    // chunks begin in the same `chunk` rows only if one is a group's first and the other is not)
    const bool whole = tab.row_off[h + 1] - tab.row_off[h] <= p.chunk;
    const float scale = whole && p.scaling ? p.scaling[h] : 1.f;
    const int64_t per = (int64_t)(p.k + p.n) * p.r;
    float* part_at = p.parts + (2 * (int64_t)(first / p.chunk) + (part == 0)) * per;
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            const int col = c0 + 16 * (CB * wave + c) + i16;
            if (col >= cols) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 16 * a + 4 * q + e;
                if (j >= p.r) continue;
                const int64_t at = of_x ? (int64_t)j * p.k + col : (int64_t)col * p.r + j;
                if (!whole) part_at[(of_x ? 0 : (int64_t)p.k * p.r) + at] = acc[a][c][e];
                else {
                    const float v = acc[a][c][e] * scale;
                    const int64_t to = (int64_t)h * (of_x ? p.k : p.n) * p.r + at;
                    void* dst = of_x ? p.da : p.db;
                    if (p.grads_bf16) Out8<uint16_t>::put((uint16_t*)dst + to, v);
                    else ((float*)dst)[to] = v;
                }
            }
        }
}

// join: groups of several chunks, in their order; groups without rows are 0
__global__ __launch_bounds__(NT) void join(Outer p, int blocks) {
    __shared__ Tables tab;
    int tiles, covered;
    build_tables<NT>(p.group_sizes, p.g, p.m, p.chunk, 1, tab, &tiles, &covered);
    const int h = blockIdx.x / blocks, b = blockIdx.x - h * blocks;
    const int first = tab.row_off[h], rows = tab.row_off[h + 1] - first;
    if (rows > 0 && rows <= p.chunk) return;
    const int chunks = (rows + p.chunk - 1) / p.chunk;
    const float scale = p.scaling ? p.scaling[h] : 1.f;
    const int64_t ka = (int64_t)p.k * p.r, per = (int64_t)(p.k + p.n) * p.r;
    for (int64_t e = (int64_t)b * NT + threadIdx.x; e < per; e += (int64_t)blocks * NT) {
        float s = 0.f;
        for (int c = 0; c < chunks; ++c) s += p.parts[(2 * (int64_t)((first + c * p.chunk) / p.chunk) + (c == 0)) * per + e];
        s *= rows > 0 ? scale : 0.f;
        if (rows == 0) s = 0.f;
        void* dst = e < ka ? p.da : p.db;
        const int64_t to = e < ka ? h * ka + e : (int64_t)h * p.n * p.r + (e - ka);
        if (p.grads_bf16) Out8<uint16_t>::put((uint16_t*)dst + to, s);
        else ((float*)dst)[to] = s;
    }
}

}  // namespace lora

// ---------------------------------------------------------------------------------------------------------------
// launches

static int64_t up64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Parts of the long axis: enough workgroups for few rows, and no part shorter than one piece of each wave.
int lora_splits(int64_t m, int64_t k) {
    const int64_t pieces = up64(k, 4 * lora::KC), want = 512 / std::max<int64_t>(1, up64(m, 16));
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(32, want), pieces));
}
// Rows that a workgroup of the row sums takes: about 1024 workgroups, and chunks long enough that their parts are few.
int lora_chunk(int64_t m, int64_t k, int64_t n) {
    const int64_t tiles = up64(k, 256) + up64(n, 256);
    const int64_t c = up64(up64(m * tiles, 1024), 32) * 32;
    return (int)std::min<int64_t>(2048, std::max<int64_t>(256, c));
}

// Rows a tile (16 MT): 64 where a group of sorted rows has that many on average.
static int lora_mt(const lora::Rows& r, int nb) {
    const int64_t rows = r.group_sizes ? r.m / r.g : std::min<int64_t>(r.m, r.chunk) / std::max(1, r.slots);
    if (nb >= 16) return 1;
    return rows >= 32 ? (nb >= 8 ? 2 : 4) : 1;
}
void lora_rows(lora::Rows& r) {
    r.chunk = (int)std::min<int64_t>(lora::MAXCHUNK, std::max<int64_t>(256, up64((int64_t)32 * r.g, 256) * 256));
    r.slots = (int)std::min<int64_t>(r.g, std::min<int64_t>(r.m, r.chunk));
}
static int64_t lora_tiles(const lora::Rows& r, int tm) {
    return r.group_sizes ? up64(r.m, tm) + r.g + 1 : std::max<int64_t>(1, up64(r.m, r.chunk)) * (r.slots + 1);
}
static int lora_nb(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : r <= 128 ? 8 : 16; }

template <typename T, int NB, int MT>
static hipError_t shrink_t(const lora::Shrink& p, hipStream_t s) {
    const int64_t tiles = lora_tiles(p.rows, 16 * MT);
    if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((lora::shrink<T, NB, MT>), dim3((uint32_t)tiles, p.splits), dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
template <typename T>
static hipError_t shrink_nb(const lora::Shrink& p, hipStream_t s) {
    const int nb = lora_nb(p.r), mt = lora_mt(p.rows, nb);
    switch (nb) {
        case 1: return mt == 1 ? shrink_t<T, 1, 1>(p, s) : shrink_t<T, 1, 4>(p, s);
        case 2: return mt == 1 ? shrink_t<T, 2, 1>(p, s) : shrink_t<T, 2, 4>(p, s);
        case 4: return mt == 1 ? shrink_t<T, 4, 1>(p, s) : shrink_t<T, 4, 4>(p, s);
        case 8: return mt == 1 ? shrink_t<T, 8, 1>(p, s) : shrink_t<T, 8, 2>(p, s);
        default: return shrink_t<T, 16, 1>(p, s);
    }
}
hipError_t launch_lora_shrink(const lora::Shrink& p, bool bf16, hipStream_t s) {
    return bf16 ? shrink_nb<uint16_t>(p, s) : shrink_nb<float>(p, s);
}

template <typename T, typename O, int NB, int MT>
static hipError_t expand_t(lora::Expand p, hipStream_t s) {
    const int64_t tiles = lora_tiles(p.rows, 16 * MT);
    p.cols = 512;
    while (p.cols > 128 && tiles * up64(p.n, p.cols) < 1024) p.cols /= 2;
    p.col_tiles = (int)std::max<int64_t>(1, up64(p.n, p.cols));
    if (tiles * p.col_tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)(tiles * p.col_tiles));
    if (p.r % 8 == 0) hipLaunchKernelGGL((lora::expand<T, O, NB, MT, true>), grid, dim3(lora::NT), 0, s, p);
    else hipLaunchKernelGGL((lora::expand<T, O, NB, MT, false>), grid, dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
template <typename T, typename O>
static hipError_t expand_nb(const lora::Expand& p, hipStream_t s) {
    const int nb = lora_nb(p.r), mt = lora_mt(p.rows, nb);
    switch (nb) {
        case 1: return mt == 1 ? expand_t<T, O, 1, 1>(p, s) : expand_t<T, O, 1, 4>(p, s);
        case 2: return mt == 1 ? expand_t<T, O, 2, 1>(p, s) : expand_t<T, O, 2, 4>(p, s);
        case 4: return mt == 1 ? expand_t<T, O, 4, 1>(p, s) : expand_t<T, O, 4, 4>(p, s);
        case 8: return mt == 1 ? expand_t<T, O, 8, 1>(p, s) : expand_t<T, O, 8, 2>(p, s);
        default: return expand_t<T, O, 16, 1>(p, s);
    }
}
hipError_t launch_lora_expand(const lora::Expand& p, bool bf16, bool out_bf16, hipStream_t s) {
    if (bf16) return out_bf16 ? expand_nb<uint16_t, uint16_t>(p, s) : expand_nb<uint16_t, float>(p, s);
    return out_bf16 ? expand_nb<float, uint16_t>(p, s) : expand_nb<float, float>(p, s);
}

hipError_t launch_lora_turn(const void* a, void* at, bool bf16, int g, int rows, int cols, hipStream_t s) {
    const int64_t tr = up64(rows, 32), tc = up64(cols, 32), blocks = tr * tc * g;
    if (blocks == 0) return hipSuccess;
    if (blocks > kMaxBlocks) return hipErrorInvalidConfiguration;
    if (bf16)
        hipLaunchKernelGGL(lora::turn<uint16_t>, dim3((uint32_t)blocks), dim3(lora::NT), 0, s, (const uint16_t*)a, (uint16_t*)at, rows, cols, (int)tr, (int)tc);
    else
        hipLaunchKernelGGL(lora::turn<float>, dim3((uint32_t)blocks), dim3(lora::NT), 0, s, (const float*)a, (float*)at, rows, cols, (int)tr, (int)tc);
    return hipGetLastError();
}

template <lora::Wide XW, int NB, int P, int CB>
static hipError_t outer_t(const lora::Outer& p, hipStream_t s) {
    const int64_t tiles = up64(p.m, p.chunk) + p.g, cols = up64(p.k, 64 * CB) + up64(p.n, 64 * CB);
    if (tiles * cols > kMaxBlocks) return hipErrorInvalidConfiguration;
    if (tiles * cols > 0) hipLaunchKernelGGL((lora::outer<XW, NB, P, CB>), dim3((uint32_t)(tiles * cols)), dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
template <lora::Wide XW, int P>
static hipError_t outer_nb(const lora::Outer& p, hipStream_t s) {
    switch (lora_nb(p.r)) {
        case 1: return outer_t<XW, 1, P, 4>(p, s);
        case 2: return outer_t<XW, 2, P, 4>(p, s);
        case 4: return outer_t<XW, 4, P, 4>(p, s);
        case 8: return outer_t<XW, 8, P, 2>(p, s);
        default: return outer_t<XW, 16, P, 1>(p, s);
    }
}
hipError_t launch_lora_outer(const lora::Outer& p, bool bf16, hipStream_t s) {
    hipError_t e;
    if (!bf16) e = outer_nb<lora::FP32, 1>(p, s);
    else if (p.x_scale) e = p.grads_bf16 ? outer_nb<lora::E4M3, 2>(p, s) : outer_nb<lora::E4M3, 3>(p, s);
    else e = p.grads_bf16 ? outer_nb<lora::BF16, 2>(p, s) : outer_nb<lora::BF16, 3>(p, s);
    if (e != hipSuccess) return e;
    const int64_t per = (int64_t)(p.k + p.n) * p.r;
    if (per == 0) return hipSuccess;
    const int blocks = (int)std::min<int64_t>(up64(per, lora::NT * 4), std::max<int64_t>(1, 4096 / p.g));
    if ((int64_t)blocks * p.g > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(lora::join, dim3((uint32_t)(blocks * p.g)), dim3(lora::NT), 0, s, p, blocks);
    return hipGetLastError();
}

}  // namespace gg
