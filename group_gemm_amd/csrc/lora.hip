// lora.hip -- low-rank adapters of many requests (or experts) at once, beside a shared projection, and their
// gradients on gfx950.  Row i of x has adapter h (its group of sorted rows, or row_group[i]), or none:
//   v[i] = x[i] . a[h]^T,   out[i] = base[i] + s[h] v[i] . b[h]^T          a [g, r, k], b [g, n, r]
//   u[i] = dout[i] . b[h],  dx[i] = dbase[i] + s[h] u[i] . a[h],
//   da[h] = s[h] sum_i u[i]^T x[i],  db[h] = s[h] sum_i dout[i]^T v[i].
// r is small beside k and n, so all of it is bound by reading x, base and dout and writing out and dx once.
//
// Three products.  `shrink` contracts the long axis (v, u): a tile of rows of one adapter against its r rows of
// weights, the axis split over workgroups where the rows are few.  `expand` contracts r and adds the other term.
// `outer` contracts the rows of a group (da, db), in chunks of rows that `join` adds up in order where a group has
// more than one: no atomics, so results do not depend on the launch.
// The backward pass is the forward one with the weights' axes swapped, so `turn` writes b as [g, r, n] and a as
// [g, k, r] once a call, which is small, and `shrink` and `expand` serve both.
// Each has a kernel for rows of whole 16 bytes (shrink_ring, expand_lines) and one or two for the rest; few rows take both
// products in one launch (`both`).  Measured, 8192 bf16 rows, 4096 x 14336, rank 64: x is read in 25 us
// (2.7 TB/s), base read and out written in 108 (4.3 TB/s; a copy reaches 4.9).
//
// Products of bf16 weights with the fp32 v and u run on the bf16 matrix instructions with v and u as a sum of two
// bf16 values (16 bits of fraction, so their error stays below a bf16 result's and 2^-17 of an fp32 one), of three
// (24 bits) in the row sums that leave in fp32.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "ring.hpp"

namespace gg {
namespace lora {

constexpr int NT = 256;
constexpr int KC = 64;           // elements of the long axis that a wave takes at a time
constexpr int MAXCHUNK = 1024;   // rows in any order: of these many, a workgroup takes those of its adapter
constexpr int NONE = 64;         // and of these many those without one

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
    // load_part in two: what is loaded past `valid`, but before `end`, the array's, is masked when all loads are on their way
    __device__ void load_tail(const uint16_t* p, int valid, const uint16_t* end) {
        if (p + 8 > end) load_part(p, valid);
        else load(p);
    }
    __device__ void mask(int valid) {
        i32x4 q = __builtin_bit_cast(i32x4, v);
#pragma unroll
        for (int d = 0; d < 4; ++d) q[d] &= valid >= 2 * d + 2 ? -1 : valid == 2 * d + 1 ? 0xffff : 0;
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
    __device__ void load_tail(const float* p, int valid, const float* end) {
        if (p + 8 > end) load_part(p, valid);
        else load(p);
    }
    __device__ void mask(int valid) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e >= valid) lo[e] = 0.f;
            if (e + 4 >= valid) hi[e] = 0.f;
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
struct RowList { int list[MAXCHUNK]; int wave[4]; };

// tile `id` of the rows behind the last adapter's
__device__ inline RowTile behind(const Rows& p, int covered, int id, int tm) {
    const int64_t first = covered + (int64_t)id * tm;
    return {-1, (int)max((int64_t)0, min((int64_t)tm, p.m - first)), (int)min(first, (int64_t)p.m), nullptr};
}
// Sorted rows: tile `id` of `tm` rows each, adapters first and then the rows behind the last one's.  Up to 64
// adapters every wave scans the sizes by itself, which takes a third of the time of the tables' two block scans.
__device__ inline RowTile sorted_tile(const Rows& p, int id, int tm, Tables& tab) {
    if (p.g <= 64) {
        const int l = threadIdx.x & 63, given = l < p.g ? p.group_sizes[l] : 0;
        uint32_t end = (uint32_t)min(max(given, 0), p.m);
        const uint32_t own = end;
        for (int d = 1; d < 64; d <<= 1) {   // sums held to m, which is associative
            const uint32_t u = (uint32_t)__shfl_up((int)end, d, 64);
            if (l >= d) end = min(end + u, (uint32_t)p.m);
        }
        uint32_t start = (uint32_t)__shfl_up((int)end, 1, 64);
        if (l == 0) start = 0;
        const int mine = (int)((end - start + tm - 1) / (uint32_t)tm);
        int tiles = mine;
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(tiles, d, 64);
            if (l >= d) tiles += u;
        }
        const int total = __shfl(tiles, 63, 64), covered = __shfl((int)end, 63, 64);
        if (p.status && blockIdx.x == 0 && blockIdx.y == 0) {
            const bool over = __any(end - start < own || (given > p.m));
            const bool negative = __any(given < 0);
            if (threadIdx.x == 0) *p.status = (negative ? GG_DEV_NEGATIVE_SIZE : 0u) | (over ? GG_DEV_SUM_EXCEEDS_M : 0u);
        }
        if (id < total) {
            const int h = __popcll(__ballot(tiles <= id));
            const int first = __shfl((int)start, h, 64) + (id - __shfl(tiles - mine, h, 64)) * tm;
            return {h, min(tm, __shfl((int)end, h, 64) - first), first, nullptr};
        }
        return behind(p, covered, id - total, tm);
    }
    int tiles, covered;
    build_tables<NT>(p.group_sizes, p.g, p.m, tm, 1, tab, &tiles, &covered);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && p.status) *p.status = tab.flags;
    RowTile w = behind(p, covered, id - tiles, tm);
    if (id < tiles) {
        const int h = find_group(tab.tile_off, p.g, id);
        const int first = tab.row_off[h] + (id - tab.tile_off[h]) * tm;
        w = {h, min(tm, tab.row_off[h + 1] - first), first, nullptr};
    }
    __syncthreads();   // the tables' memory is used again
    return w;
}
// Rows in any order: slot `id` of a chunk is adapter `id`, or (fewer rows than adapters) the adapter of row `id` of
// the chunk if no row before it has the same; the last slots are the rows without one, of
// NONE rows each.  The list is in row order.
__device__ inline RowTile any_tile(const Rows& p, int id, RowList& any) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && p.status) *p.status = 0;
    const int slots = p.slots + p.chunk / NONE, c = id / slots, slot = id - c * slots;
    int r0 = c * p.chunk, n = min(p.chunk, p.m - r0);
    const bool by_row = p.slots < p.g;
    int h = slot;
    if (slot >= p.slots) {
        h = -1;
        r0 += (slot - p.slots) * NONE;
        n = min(NONE, p.m - r0);
        if (slot - p.slots >= p.chunk / NONE || n <= 0) return {-1, 0, 0, nullptr};
    } else if (by_row) {
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
        if ((t & 63) == 0) any.wave[w] = __popcll(mine);
        __syncthreads();
        int at = found;
        for (int j = 0; j < 4; ++j) {
            if (j < w) at += any.wave[j];
            found += any.wave[j];
        }
        if (of == h) any.list[at + __popcll(mine & ((1ull << (t & 63)) - 1))] = r0 + i;
        __syncthreads();
    }
    if (by_row && h >= 0 && found > 0 && any.list[0] != r0 + slot) found = 0;   // an earlier row's slot has them
    return {h, found, 0, any.list};
}
// `scratch`: LDS that is free until the call returns
__device__ inline RowTile row_tile(const Rows& p, int id, int tm, RowList& any, void* scratch) {
    return p.group_sizes ? sorted_tile(p, id, tm, *(Tables*)scratch) : any_tile(p, id, any);
}
__device__ inline int row_at(const RowTile& w, int i) { return w.list ? w.list[i] : w.first + i; }

// ---------------------------------------------------------------------------------------------------------------
// shrink: t[split, row, j] = x[row] . w[h][j], over the split's part of the long axis.  16 rows, 16 NB columns j.
// The weights are the first operand, so a lane ends with four consecutive j of one row.  This one is for few rows of any
// alignment: the four waves take the axis in turn, fragments come straight from memory.

template <typename T, int NB, int U>   // U pieces of the axis in flight
__global__ __launch_bounds__(NT) void shrink(Shrink p) {
    constexpr int TM = 16;
    __shared__ RowList rs;
    __shared__ union { f32x4 red[2][NB * 64]; Tables tab; } sm;
    auto& red = sm.red;
    const RowTile w = row_tile(p.rows, blockIdx.x, TM, rs, &sm);
    if (w.h < 0 || w.rows == 0) return;
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;
    const int nch = (p.k + KC - 1) / KC, per = (nch + (int)gridDim.y - 1) / (int)gridDim.y;
    const int c0 = blockIdx.y * per, c1 = min(nch, c0 + per);
    const T* wp[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wp[b] = (const T*)p.w + ((int64_t)w.h * p.r + min(16 * b + i16, p.r - 1)) * p.k + 8 * q;
    for (int r0 = 0; r0 < w.rows; r0 += TM) {
        const T* xp = (const T*)p.x + (int64_t)row_at(w, min(r0 + i16, w.rows - 1)) * p.stride + 8 * q;
        f32x4 acc[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int whole = min(c1, p.k / KC);   // chunks that lie inside the axis
        auto pieces = [&](int c, auto u_c) {
            constexpr int N = decltype(u_c)::value;
            Frag<T> x[N][2], m[N][2][NB];
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    x[u][s].load(xp + (int64_t)(c + 4 * u) * KC + 32 * s);
#pragma unroll
                    for (int b = 0; b < NB; ++b) m[u][s][b].load(wp[b] + (int64_t)(c + 4 * u) * KC + 32 * s);
                }
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[b] = Frag<T>::mma(m[u][s][b], x[u][s], acc[b]);
        };
        int c = c0 + wave;
        for (; c + 4 * (U - 1) < whole; c += 4 * U) pieces(c, std::integral_constant<int, U>{});
        if constexpr (U > 1)
            for (; c < whole; c += 4) pieces(c, std::integral_constant<int, 1>{});
        if (c0 <= whole && whole < c1 && (whole - c0) % 4 == wave) {   // the chunk that the axis ends in
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int valid = p.k - whole * KC - 32 * s - 8 * q;
                Frag<T> x, m[NB];
                x.load_part(xp + (int64_t)whole * KC + 32 * s, valid);
#pragma unroll
                for (int b = 0; b < NB; ++b) m[b].load_part(wp[b] + (int64_t)whole * KC + 32 * s, valid);
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[b] = Frag<T>::mma(m[b], x, acc[b]);
            }
        }
        // waves 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
        for (int half = 2; half >= 1; half >>= 1) {
            if (wave >= half && wave < 2 * half)
#pragma unroll
                for (int b = 0; b < NB; ++b) red[wave - half][b * 64 + l] = acc[b];
            __syncthreads();
            if (wave < half)
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[b] += red[wave][b * 64 + l];
            __syncthreads();
        }
        if (wave == 0 && r0 + i16 < w.rows) {
            float* to = p.t + ((int64_t)blockIdx.y * p.rows.m + row_at(w, r0 + i16)) * p.r;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 16 * b + 4 * q + e;
                    if (j < p.r) to[j] = acc[b][e];
                }
        }
    }
}

// The same through LDS, for rows of whole 16 bytes.  A matrix instruction's lanes 0 .. 15 hold sixteen rows, so fragments
// loaded straight from memory touch a line a lane, and the address path, not the memory, sets the pace (3 TB/s at rank
// 16, 1.5 at rank 64).  Here eight lanes load 128 contiguous bytes of a row straight into LDS, in a ring of D slots, and
// the fragments come from there.  A slot is [rows][128 bytes], its 16-byte pieces XOR'ed with the row so that a
// fragment's lanes read from all banks.  TEAM = 4: the four waves share one ring and the weights in it, 16 rows each;
// TEAM = 1 (few rows an adapter): each wave has a ring of its own, the pieces of the axis are dealt to the waves, and no
// barrier is needed until their sums are added up.
template <typename T> __device__ inline Frag<T> ring_frag(const char* slot, int row, int s);
template <> __device__ inline Frag<uint16_t> ring_frag<uint16_t>(const char* slot, int row, int s) {
    const int q = (threadIdx.x & 63) >> 4;
    Frag<uint16_t> f;
    f.v = *(const bf16x8*)(slot + row * 128 + 16 * ((4 * s + q) ^ ((row >> 1) & 7)));
    return f;
}
template <> __device__ inline Frag<float> ring_frag<float>(const char* slot, int row, int) {
    const int q = (threadIdx.x & 63) >> 4;
    Frag<float> f;
    f.lo = *(const f32x4*)(slot + row * 128 + 16 * ((2 * q) ^ ((row >> 1) & 7)));
    f.hi = *(const f32x4*)(slot + row * 128 + 16 * ((2 * q + 1) ^ ((row >> 1) & 7)));
    return f;
}
// 16 bytes a lane from memory straight into LDS at lds + 16 * lane, outside the compiler's wait tracking (ring.hpp)
__device__ inline void load_lds16_at(const char* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(lds), "v"(p) : "memory", "m0");
}

// One tile of rows r0 .. of a ring: on return `acc` is the wave's 16 rows' (TEAM = 4) or, in wave 0, the 16 rows' sums
// over the pieces c0 .. c1 - 1 of the axis.  All waves call it together; the rings may be used again after a barrier.
template <typename T, int NB, int TEAM, int D> struct Ring {
    static constexpr int TM = 16 * TEAM, WB = TEAM == 4 && NB < 2 ? 2 : NB;   // rows; blocks of 16 weight rows in a slot
    static constexpr int SLOT = (TM + 16 * WB) * 128, PER = (TM + 16 * WB) / 8 / TEAM;   // bytes; loads a wave
    static constexpr int KE = 128 / sizeof(T), STEPS = sizeof(T) == 2 ? 2 : 1, RINGS = 4 / TEAM, BYTES = RINGS * D * SLOT;
    static_assert(PER * (D - 1) <= 63, "vmcnt range");
    static_assert(BYTES >= (RINGS > 1 ? 2 * NB * 64 * 16 : 0), "the sums of the waves fit the rings");
    static_assert(BYTES >= (int)sizeof(Tables), "the rings hold the tables first");
    __device__ static void run(f32x4 (&acc)[NB], char* rings, const Shrink& p, const RowTile& w, int r0, int c0, int c1) {
        const int t = threadIdx.x, l = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), q = l >> 4, i16 = l & 15;
        const int mate = TEAM == 4 ? wave : 0, alone = TEAM == 4 ? 0 : wave;
        const int whole = min(c1, p.k / KE);
        const int count = max(0, whole - c0 - alone + (RINGS - 1)) / RINGS;   // this ring's pieces: every RINGS-th
        const char* ring = rings + alone * (D * SLOT);
        const uint32_t lds = ring::lds_u32(ring);
        // load u of this wave: rows 8 (PER mate + u) .. + 7 of the slot, x's first and then the weights'
        const char* src[PER];
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int row = 8 * (PER * mate + u) + (l >> 3), piece = 16 * ((l & 7) ^ ((row >> 1) & 7));
            const T* at = row < TM ? (const T*)p.x + (int64_t)row_at(w, min(r0 + row, w.rows - 1)) * p.stride
                                   : (const T*)p.w + ((int64_t)w.h * p.r + min(row - TM, p.r - 1)) * p.k;
            src[u] = (const char*)(at + (int64_t)(c0 + alone) * KE) + piece;
        }
        auto issue = [&](int i, int slot) {   // past the end: the last piece again, which no one reads
            const int64_t off = (int64_t)min(i, count - 1) * (RINGS * 128);
#pragma unroll
            for (int u = 0; u < PER; ++u)
                load_lds16_at(src[u] + off, __builtin_amdgcn_readfirstlane(lds + slot * SLOT + (PER * mate + u) * 1024));
        };
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (count > 0) {
#pragma unroll
            for (int d = 0; d < D - 1; ++d) issue(d, d);
            int slot = 0;
            for (int i = 0; i < count; ++i) {
                ring::wait_vm<PER * (D - 2)>();   // piece i is in LDS: this wave's part of it
                if (TEAM == 4) ring::lds_barrier();   // and the others'; and piece i - 1 has been read
                const char* at = ring + slot * SLOT;
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const Frag<T> x = ring_frag<T>(at, 16 * mate + i16, s);
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[b] = Frag<T>::mma(ring_frag<T>(at, TM + 16 * b + i16, s), x, acc[b]);
                }
                if (TEAM == 1) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // a wave alone: its reads are done
                issue(i + D - 1, slot == 0 ? D - 1 : slot - 1);
                slot = slot == D - 1 ? 0 : slot + 1;
            }
        }
        ring::wait_vm<0>();
        if (c0 <= whole && whole < c1 && (TEAM == 4 || (whole - c0) % RINGS == wave)) {   // the piece that the axis ends in
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int e0 = whole * KE + 32 * s + 8 * q, valid = p.k - e0;
                Frag<T> x;
                x.load_part((const T*)p.x + (int64_t)row_at(w, min(r0 + 16 * mate + i16, w.rows - 1)) * p.stride + e0, valid);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    Frag<T> m;
                    m.load_part((const T*)p.w + ((int64_t)w.h * p.r + min(16 * b + i16, p.r - 1)) * p.k + e0, valid);
                    acc[b] = Frag<T>::mma(m, x, acc[b]);
                }
            }
        }
        if constexpr (RINGS > 1) {   // waves 2 and 3 to 0 and 1, then 1 to 0
            f32x4* red = (f32x4*)rings;
            __syncthreads();
#pragma unroll
            for (int half = 2; half >= 1; half >>= 1) {
                if (wave >= half && wave < 2 * half)
#pragma unroll
                    for (int b = 0; b < NB; ++b) red[((wave - half) * NB + b) * 64 + l] = acc[b];
                __syncthreads();
                if (wave < half)
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[b] += red[(wave * NB + b) * 64 + l];
                __syncthreads();
            }
        }
    }
};

template <typename T, int NB, int TEAM, int D>
__global__ __launch_bounds__(NT) void shrink_ring(Shrink p) {
    using R = Ring<T, NB, TEAM, D>;
    __shared__ RowList rs;
    __shared__ __attribute__((aligned(128))) char rings[R::BYTES];
    const RowTile w = row_tile(p.rows, blockIdx.x, R::TM, rs, rings);
    if (w.h < 0 || w.rows == 0) return;
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, q = l >> 4;
    const int nch = (p.k + R::KE - 1) / R::KE, per = (nch + (int)gridDim.y - 1) / (int)gridDim.y;
    const int c0 = blockIdx.y * per, c1 = min(nch, c0 + per);
    for (int r0 = 0; r0 < w.rows; r0 += R::TM) {
        if (r0 > 0 || w.list) ring::lds_barrier();   // the list and the last tile's sums have been read
        f32x4 acc[NB];
        R::run(acc, rings, p, w, r0, c0, c1);
        const int row = r0 + (TEAM == 4 ? 16 * wave : 0) + (l & 15);
        if ((TEAM == 1 && wave > 0) || row >= w.rows) continue;
        float* to = p.t + ((int64_t)blockIdx.y * p.rows.m + row_at(w, row)) * p.r;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (16 * b + 4 * q + e < p.r) to[16 * b + 4 * q + e] = acc[b][e];
    }
}

// The same for many rows of any alignment: 64 rows a workgroup, through registers (loads straight into LDS take whole
// dwords), two pieces on their way.
template <typename T, int NB>
__global__ __launch_bounds__(NT) void shrink_staged(Shrink p) {
    constexpr int TM = 64, KE = 128 / sizeof(T), STEPS = sizeof(T) == 2 ? 2 : 1, EL = 16 / sizeof(T);
    constexpr int ROWS = TM + 16 * NB, PER = (ROWS + 31) / 32;   // rows of a slot; 16-byte loads a thread
    __shared__ RowList rs;
    __shared__ union { Tables tab; __attribute__((aligned(128))) char slot[2][PER * 32 * 128]; } sm;
    const RowTile w = row_tile(p.rows, blockIdx.x, TM, rs, &sm);
    if (w.h < 0 || w.rows == 0) return;
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;
    const int nch = (p.k + KE - 1) / KE, per = (nch + (int)gridDim.y - 1) / (int)gridDim.y;
    const int c0 = blockIdx.y * per, c1 = min(nch, c0 + per);
    for (int r0 = 0; r0 < w.rows; r0 += TM) {
        const T* src[PER];
        int at[PER];
#pragma unroll
        for (int u = 0; u < PER; ++u) {   // row t / 8 + 32 u of a slot, x's first and then the weights', 16 bytes of it
            const int row = (t >> 3) + 32 * u;
            src[u] = (row < TM ? (const T*)p.x + (int64_t)row_at(w, min(r0 + row, w.rows - 1)) * p.stride
                               : (const T*)p.w + ((int64_t)w.h * p.r + min(row - TM, p.r - 1)) * p.k) + EL * (t & 7);
            at[u] = row * 128 + 16 * ((t & 7) ^ ((row >> 1) & 7));
        }
        i32x4 v[2][PER];
        auto load = [&](i32x4 (&to)[PER], int c) {
            const int valid = min(p.k - c * KE - EL * (t & 7), EL);   // of the thread's elements
            if (c >= c1) return;
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                if (valid == EL) to[u] = *(const i32x4_any*)(src[u] + (int64_t)c * KE);
                else {
                    to[u] = i32x4{0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < EL; ++e)
                        if (e < valid) {
                            if constexpr (sizeof(T) == 2) to[u][e >> 1] |= (int)((uint32_t)src[u][(int64_t)c * KE + e] << (16 * (e & 1)));
                            else to[u][e] = __float_as_int(src[u][(int64_t)c * KE + e]);
                        }
                }
            }
        };
        f32x4 acc[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto step = [&](auto z_c, int c) {
            constexpr int z = decltype(z_c)::value;
#pragma unroll
            for (int u = 0; u < PER; ++u) *(i32x4*)(sm.slot[z] + at[u]) = v[z][u];
            load(v[z], c + 2);
            __syncthreads();   // the other slot is written only after every wave has passed this, its reads done
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const Frag<T> x = ring_frag<T>(sm.slot[z], 16 * wave + i16, s);
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[b] = Frag<T>::mma(ring_frag<T>(sm.slot[z], TM + 16 * b + i16, s), x, acc[b]);
            }
        };
        __syncthreads();       // the list, and the last tile's slots, have been read
        load(v[0], c0);
        load(v[1], c0 + 1);
        for (int c = c0; c < c1; c += 2) {
            step(std::integral_constant<int, 0>{}, c);
            if (c + 1 < c1) step(std::integral_constant<int, 1>{}, c + 1);
        }
        const int row = r0 + 16 * wave + i16;
        if (row >= w.rows) continue;
        float* to = p.t + ((int64_t)blockIdx.y * p.rows.m + row_at(w, row)) * p.r;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (16 * b + 4 * q + e < p.r) to[16 * b + 4 * q + e] = acc[b][e];
    }
}

// ---------------------------------------------------------------------------------------------------------------
// expand: out[row] = base[row] + s[h] t[row] . w[h]^T for 16 MT rows and `cols` columns, t being the sum of the
// splits.  The weights are the first operand, so a lane ends with four columns of one row, and consecutive lanes with
// different rows; results turn in LDS so that eight lanes read 128 contiguous bytes of base and write them of out.

// `hold`: rows whose ends share lines with their neighbours are stored so that the caches may wait for the rest of a line
// (8192 rows of 4095 bf16 columns 57 us against 45); whole lines leave at once (4096 fp32 columns 111 us against 121).
template <typename O> struct Out8;
template <> struct Out8<uint16_t> {
    i32x4 q;
    __device__ void load(const uint16_t* p) { q = *(const i32x4_any*)p; }
    __device__ float get(int i) const { return __uint_as_float((i & 1) ? (uint32_t)q[i >> 1] & 0xffff0000u : (uint32_t)q[i >> 1] << 16); }
    __device__ void zero() { q = i32x4{0, 0, 0, 0}; }
    __device__ static float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
    __device__ static void put(uint16_t* p, float v) { const __bf16 b = (__bf16)v; *p = __builtin_bit_cast(uint16_t, b); }
    __device__ static void store(uint16_t* p, const float (&v)[8], bool hold) {
        i32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
            w[i] = __builtin_bit_cast(int, b);
        }
        if (hold) *(i32x4_any*)p = w;
        else __builtin_nontemporal_store(w, (i32x4_any*)p);
    }
};
template <> struct Out8<float> {
    f32x4 a, b;
    __device__ void load(const float* p) {
        a = *(const f32x4_any*)p;
        b = *(const f32x4_any*)(p + 4);
    }
    __device__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
    __device__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ static float one(const float* p) { return *p; }
    __device__ static void put(float* p, float v) { *p = v; }
    __device__ static void store(float* p, const float (&v)[8], bool hold) {
        const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        if (hold) {
            *(f32x4_any*)p = a;
            *(f32x4_any*)(p + 4) = b;
        } else {
            __builtin_nontemporal_store(a, (f32x4_any*)p);
            __builtin_nontemporal_store(b, (f32x4_any*)(p + 4));
        }
    }
};

// t of a tile's rows as the second operand, in steps of 32 elements of r: bf16 [high | low], fp32 as it is.
template <typename T, int NB> struct Narrow {
    static constexpr int STEPS = NB < 2 ? 1 : NB / 2, PARTS = sizeof(T) == 2 ? 2 : 1;
    static constexpr int PITCH = PARTS * 32 * STEPS + (sizeof(T) == 2 ? 8 : 4);
};

// Columns col0 .. col1 - 1 of rows r0 .. of a tile, whose t is in `nar`; a strip of 16 rows of 64 columns a wave turns
// results into whole lines.
constexpr int SP = 64 + 4;
struct Strips { __attribute__((aligned(16))) float of[4][16 * SP]; };
template <typename T, typename O, int NB, int MT, bool WHOLE>   // WHOLE: r % 8 == 0
__device__ inline void columns(const Expand& p, const RowTile& w, int r0, int col0, int col1, const T* nar, Strips& strips) {
    using N = Narrow<T, NB>;
    constexpr int PITCH = N::PITCH, STEPS = N::STEPS, PARTS = N::PARTS;
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;
    const O* base = (const O*)p.base;
    O* out = (O*)p.out;
    const int last = (p.r + 7) / 8 - 1;                 // the last eight of r
    const T* wb = (const T*)p.w + (int64_t)w.h * p.n * p.r;
    const bool hold = p.out_stride * sizeof(O) % 16 != 0 || (uintptr_t)p.out % 16 != 0;
    // a wave: 64 columns of all rows at a time, the next ones' base on its way
    auto fetch = [&](Out8<O> (&o)[MT][2], int c) {
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const int i = r0 + 16 * a + 8 * d + (l >> 3), cc = c + 8 * (l & 7);
                o[a][d].zero();
                if (base && i < w.rows && cc + 8 <= col1) o[a][d].load(base + (int64_t)row_at(w, i) * p.base_stride + cc);
            }
    };
    Out8<O> next[MT][2];
    fetch(next, col0 + 64 * wave);
    for (int c = col0 + 64 * wave; c < col1; c += 256) {
        Out8<O> o[MT][2];
#pragma unroll
        for (int a = 0; a < MT; ++a) { o[a][0] = next[a][0]; o[a][1] = next[a][1]; }
        Frag<T> m[4][STEPS];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const T* wr = wb + (int64_t)min(c + 16 * j + i16, p.n - 1) * p.r;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int e = 8 * min(4 * s + q, last);   // past the end: times the zeros above
                if (WHOLE) m[j][s].load(wr + e);
                else m[j][s].load_tail(wr + e, p.r - e, (const T*)p.w + (int64_t)p.rows.g * p.n * p.r);
            }
        }
        fetch(next, c + 256);
        if constexpr (!WHOLE) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < STEPS; ++s) m[j][s].mask(p.r - 8 * min(4 * s + q, last));
        }
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            f32x4 acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int z = 0; z < PARTS; ++z) {
                    Frag<T> x;
                    x.load_lds(nar + (16 * a + i16) * PITCH + 32 * (STEPS * z + s) + 8 * q);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[j] = Frag<T>::mma(m[j][s], x, acc[j]);
                }
            float* strip = strips.of[wave];
#pragma unroll
            for (int j = 0; j < 4; ++j) *(f32x4*)(strip + i16 * SP + 16 * j + 4 * q) = acc[j];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const int i = r0 + 16 * a + 8 * d + (l >> 3), cc = c + 8 * (l & 7);
                const float* from = strip + (8 * d + (l >> 3)) * SP + 8 * (l & 7);
                const f32x4 lo = *(const f32x4*)from, hi = *(const f32x4*)(from + 4);
                if (i >= w.rows || cc >= col1) continue;
                const int64_t row = row_at(w, i);
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) { v[e] = lo[e]; v[4 + e] = hi[e]; }
                if (cc + 8 <= p.n) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += o[a][d].get(e);
                    Out8<O>::store(out + row * p.out_stride + cc, v, hold);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (cc + e < p.n)
                            Out8<O>::put(out + row * p.out_stride + cc + e, v[e] + (base ? Out8<O>::one(base + row * p.base_stride + cc + e) : 0.f));
                }
            }
        }
    }
}
// rows without an adapter: what was there.  E: what moves at once, O or whole 16 bytes of it; eight of a thread in flight
template <typename O, typename E>
__device__ inline void untouched(const Expand& p, const RowTile& w, int ct, int col0, int col1) {
    constexpr int PER = sizeof(E) / sizeof(O);
    if (p.v && ct == 0)
        for (int e = threadIdx.x; e < w.rows * p.r; e += NT) p.v[(int64_t)row_at(w, e / p.r) * p.r + e % p.r] = 0.f;
    if ((p.base == p.out && p.base_stride == p.out_stride) || col1 <= col0) return;
    const uint32_t width = (uint32_t)(col1 - col0) / PER, total = (uint32_t)w.rows * width;
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += 8 * NT) {
        E v[8];
        int64_t to[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t e = min(e0 + NT * u, total - 1), i = e / width, c = (e - i * width) * PER + col0;
            const int64_t row = row_at(w, (int)i);
            to[u] = row * p.out_stride + c;
            v[u] = p.base ? *(const E*)((const O*)p.base + row * p.base_stride + c) : E{};
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (e0 + NT * u < total) *(E*)((O*)p.out + to[u]) = v[u];
    }
}

template <typename T, typename O, int NB, int MT, bool WHOLE>   // WHOLE: r % 8 == 0
__global__ __launch_bounds__(NT) void expand(Expand p) {
    using N = Narrow<T, NB>;
    constexpr int TM = 16 * MT, PITCH = N::PITCH, STEPS = N::STEPS, PARTS = N::PARTS;
    __shared__ RowList rs;
    __shared__ __attribute__((aligned(16))) T nar[TM * PITCH];
    __shared__ Strips strips;
    const int ct = blockIdx.x % p.col_tiles, id = blockIdx.x / p.col_tiles;
    static_assert(sizeof(strips) >= sizeof(Tables), "the strips hold the tables first");
    const RowTile w = row_tile(p.rows, id, TM, rs, &strips);
    const int t = threadIdx.x;
    const int col0 = ct * p.cols, col1 = min(p.n, col0 + p.cols);
    if (w.h < 0) { untouched<O, O>(p, w, ct, col0, col1); return; }
    const float scale = p.scaling ? p.scaling[w.h] : 1.f;
    for (int r0 = 0; r0 < w.rows; r0 += TM) {
        if (r0) __syncthreads();
        for (int e0 = 0; e0 < TM * 32 * STEPS; e0 += 8 * NT) {   // t: eight values of a thread in flight
            constexpr int NE = TM * 32 * STEPS < 8 * NT ? TM * 32 * STEPS / NT : 8;
            float sum[NE];
            int64_t from[NE];
            bool have[NE];
#pragma unroll
            for (int u = 0; u < NE; ++u) {
                const int e = e0 + t + NT * u, i = e / (32 * STEPS), j = e % (32 * STEPS);   // (powers of two)
                have[u] = r0 + i < w.rows && j < p.r;
                from[u] = have[u] ? (int64_t)row_at(w, r0 + i) * p.r + j : 0;
                sum[u] = 0.f;
            }
            for (int k = 0; k < p.splits; k += 4) {   // four parts at a time, added in order
                float f[4][NE];
#pragma unroll
                for (int z = 0; z < 4; ++z)
#pragma unroll
                    for (int u = 0; u < NE; ++u) f[z][u] = k + z < p.splits ? p.t[(int64_t)(k + z) * p.rows.m * p.r + from[u]] : 0.f;
#pragma unroll
                for (int z = 0; z < 4; ++z)
#pragma unroll
                    for (int u = 0; u < NE; ++u) sum[u] += f[z][u];
            }
#pragma unroll
            for (int u = 0; u < NE; ++u) {
                const int e = e0 + t + NT * u, i = e / (32 * STEPS), j = e % (32 * STEPS);
                if (!have[u]) sum[u] = 0.f;
                if (have[u] && p.v && ct == 0 && p.v != p.t) p.v[from[u]] = sum[u];
                if constexpr (PARTS == 2) {
                    uint16_t two[2];
                    split<2>(sum[u] * scale, two);
                    nar[i * PITCH + j] = two[0];
                    nar[i * PITCH + 32 * STEPS + j] = two[1];
                } else {
                    nar[i * PITCH + j] = sum[u] * scale;
                }
            }
        }
        __syncthreads();
        columns<T, O, NB, MT, WHOLE>(p, w, r0, col0, col1, nar, strips);
    }
}

// Both products of few rows an adapter in one launch: a workgroup contracts the whole long axis of its 16 rows by itself
// and then takes its columns.  The first weights are read once for every `cols` columns, from L2, and there is no second
// launch to wait for and no t in memory.
struct Both { Shrink s; Expand e; };
template <typename T, typename O, int NB, int D, bool WHOLE>
__global__ __launch_bounds__(NT) void both(Both b) {
    using R = Ring<T, NB, 1, D>;
    using N = Narrow<T, NB>;
    constexpr int PITCH = N::PITCH, STEPS = N::STEPS;
    __shared__ RowList rs;
    struct After { float t[16][16 * NB + 4]; __attribute__((aligned(16))) T nar[16 * PITCH]; Strips strips; };
    __shared__ __attribute__((aligned(128))) char rings[R::BYTES > (int)sizeof(After) ? R::BYTES : sizeof(After)];
    const Expand& p = b.e;
    const int ct = blockIdx.x % p.col_tiles, id = blockIdx.x / p.col_tiles;
    const RowTile w = row_tile(p.rows, id, 16, rs, rings);
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4;
    const int col0 = ct * p.cols, col1 = min(p.n, col0 + p.cols);
    if (w.h < 0) { untouched<O, O>(p, w, ct, col0, col1); return; }
    const float scale = p.scaling ? p.scaling[w.h] : 1.f;
    After& a = *(After*)rings;
    for (int r0 = 0; r0 < w.rows; r0 += 16) {
        __syncthreads();
        f32x4 acc[NB];
        R::run(acc, rings, b.s, w, r0, 0, (b.s.k + R::KE - 1) / R::KE);
        if (wave == 0)
#pragma unroll
            for (int i = 0; i < NB; ++i) *(f32x4*)&a.t[l & 15][16 * i + 4 * q] = acc[i];
        __syncthreads();
        for (int e = t; e < 16 * 32 * STEPS; e += NT) {
            const int i = e / (32 * STEPS), j = e % (32 * STEPS);
            const bool have = r0 + i < w.rows && j < p.r;
            const float s = have ? a.t[i][j] : 0.f;
            if (have && p.v && ct == 0) p.v[(int64_t)row_at(w, r0 + i) * p.r + j] = s;
            if constexpr (N::PARTS == 2) {
                uint16_t two[2];
                split<2>(s * scale, two);
                a.nar[i * PITCH + j] = two[0];
                a.nar[i * PITCH + 32 * STEPS + j] = two[1];
            } else {
                a.nar[i * PITCH + j] = s * scale;
            }
        }
        __syncthreads();
        columns<T, O, NB, 1, WHOLE>(p, w, r0, col0, col1, a.nar, a.strips);
    }
}

// The same for many rows of bf16 weights, rows of whole 16 bytes and ranks of whole eights: 64 MT rows a workgroup, 16 MT a
// wave.  All four waves multiply with the same 64 columns' weights, which lie together in memory, so they are loaded as
// whole lines, once a workgroup, into one of two LDS slots (fragments straight from memory touch a line a lane, and their
// loads set the pace of the kernel above: 470 MB at rank 64 took 137 us).  t stays in registers.  Base, the weights two
// steps on and the results are loaded and stored without branches (offsets outside their descriptor read as 0 and are not
// stored), so no wait counts on fewer operations in flight than there are, and none waits for stores just issued.
template <typename O> struct Line8;
template <> struct Line8<uint16_t> {
    i32x4 q;
    __device__ void load(ring::rsrc_t r, uint32_t off) { q = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 2); }
    __device__ float get(int i) const { return __uint_as_float((i & 1) ? (uint32_t)q[i >> 1] & 0xffff0000u : (uint32_t)q[i >> 1] << 16); }
    __device__ static void store(ring::rsrc_t r, uint32_t off, const float (&v)[8]) {
        ring::bstore(r, off, i32x4{(int)ring::pack_bf16(v[0], v[1]), (int)ring::pack_bf16(v[2], v[3]), (int)ring::pack_bf16(v[4], v[5]),
                                   (int)ring::pack_bf16(v[6], v[7])});
    }
};
template <> struct Line8<float> {
    i32x4 a, b;
    __device__ void load(ring::rsrc_t r, uint32_t off) {
        a = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 2);
        b = __builtin_amdgcn_raw_buffer_load_b128(r, off, 16, 2);
    }
    __device__ float get(int i) const { return __int_as_float(i < 4 ? a[i] : b[i - 4]); }
    __device__ static void store(ring::rsrc_t r, uint32_t off, const float (&v)[8]) {
        ring::bstore(r, off, i32x4{__float_as_int(v[0]), __float_as_int(v[1]), __float_as_int(v[2]), __float_as_int(v[3])});
        ring::bstore(r, off + 16, i32x4{__float_as_int(v[4]), __float_as_int(v[5]), __float_as_int(v[6]), __float_as_int(v[7])});
    }
};

template <typename O, int NB, int MT>
__global__ __launch_bounds__(NT) void expand_lines(Expand p) {
    constexpr int STEPS = NB < 2 ? 1 : NB / 2, TM = 64 * MT, PITCH = 64 * STEPS + 8;   // PITCH: [high | low] of a row of t
    constexpr int ROWB = 64 * STEPS, SLOT = 64 * ROWB;           // bytes of a column's weights, of 64 columns'
    constexpr int WL = (64 * 2 * NB + NT - 1) / NT;              // 16-byte loads a thread of 64 columns' weights
    __shared__ union {
        Tables tab;
        __attribute__((aligned(16))) uint16_t nar[TM * PITCH];
        struct { __attribute__((aligned(16))) char w[2][SLOT]; __attribute__((aligned(16))) float strips[4][16 * SP]; } s;
    } sm;
    __shared__ RowList rs;
    const int ct = blockIdx.x % p.col_tiles, id = blockIdx.x / p.col_tiles;
    const RowTile w = row_tile(p.rows, id, TM, rs, &sm);
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;
    const int col0 = ct * p.cols, col1 = min(p.n, col0 + p.cols);
    constexpr uint32_t os = sizeof(O);
    if (w.h < 0) { untouched<O, i32x4>(p, w, ct, col0, col1); return; }
    const float scale = p.scaling ? p.scaling[w.h] : 1.f;
    const int pieces = p.r / 8;                                  // 16-byte pieces of a column's weights
    const ring::rsrc_t rw = ring::make_rsrc((const uint16_t*)p.w + (int64_t)w.h * p.n * p.r, (uint32_t)p.n * p.r * 2u);
    // where the thread's pieces of 64 columns' weights lie in a slot (rows of ROWB bytes, XOR'ed so that the 16 lanes of a
    // fragment read from all banks), -1: none
    int at[WL];
#pragma unroll
    for (int u = 0; u < WL; ++u) {
        const int e = t + NT * u, col = e / pieces;
        at[u] = e < 64 * pieces ? col * ROWB + 16 * ((e - col * pieces) ^ (STEPS == 1 ? (col >> 2) & 3 : STEPS == 2 ? (col >> 1) & 7 : col & 15)) : -1;
    }
    auto slot_frag = [&](const char* slot, int col, int s) {
        const int x = STEPS == 1 ? (col >> 2) & 3 : STEPS == 2 ? (col >> 1) & 7 : col & 15;
        return *(const bf16x8*)(slot + col * ROWB + 16 * ((4 * s + q) ^ x));
    };
    for (int r0 = 0; r0 < w.rows; r0 += TM) {
        __syncthreads();
        {   // t: four values a load, all of a thread's in flight
            constexpr int NE = TM * 8 * STEPS / NT;
            f32x4 sum[NE];
            int64_t from[NE];
            bool have[NE];
#pragma unroll
            for (int u = 0; u < NE; ++u) {
                const int i = (t + NT * u) / (8 * STEPS), j = 4 * ((t + NT * u) % (8 * STEPS));
                have[u] = r0 + i < w.rows && j < p.r;
                from[u] = have[u] ? (int64_t)row_at(w, r0 + i) * p.r + j : 0;
                sum[u] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            for (int k = 0; k < p.splits; ++k) {
                const float* part = p.t + (int64_t)k * p.rows.m * p.r;
                f32x4 f[NE];
#pragma unroll
                for (int u = 0; u < NE; ++u) f[u] = *(const f32x4_any*)(part + from[u]);
#pragma unroll
                for (int u = 0; u < NE; ++u) sum[u] += f[u];
            }
            const bool keep = p.v && ct == 0 && p.v != p.t;
#pragma unroll
            for (int u = 0; u < NE; ++u) {
                if (!have[u]) sum[u] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (keep && have[u]) *(f32x4_any*)(p.v + from[u]) = sum[u];
                const int i = (t + NT * u) / (8 * STEPS), j = 4 * ((t + NT * u) % (8 * STEPS));
                uint16_t two[4][2];
#pragma unroll
                for (int e = 0; e < 4; ++e) split<2>(sum[u][e] * scale, two[e]);
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    *(i32x2*)(sm.nar + i * PITCH + 32 * STEPS * z + j) = i32x2{two[0][z] | two[1][z] << 16, two[2][z] | two[3][z] << 16};
            }
        }
        __syncthreads();
        bf16x8 x[MT][STEPS][2];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int z = 0; z < 2; ++z) x[a][s][z] = *(const bf16x8*)(sm.nar + (16 * (MT * wave + a) + i16) * PITCH + 32 * (STEPS * z + s) + 8 * q);
        __syncthreads();
        // a slot's pieces past r are multiplied with zeros of t: they have to be finite
        for (int e = t; e < 2 * SLOT / 16; e += NT) *(i32x4*)(&sm.s.w[0][0] + 16 * e) = i32x4{0, 0, 0, 0};
        // rows of the tile from its first row (a chunk's, in any order): offsets stay in 32 bits
        const int64_t top = w.list ? (int64_t)w.list[0] : w.first + r0;
        const ring::rsrc_t rb = ring::make_rsrc((const O*)p.base + top * p.base_stride, p.base ? 0x7fffffffu : 0u);
        const ring::rsrc_t ro = ring::make_rsrc((O*)p.out + top * p.out_stride, 0x7fffffffu);
        uint32_t bo[MT][2], oo[MT][2];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const int i = r0 + 16 * (MT * wave + a) + 8 * d + (l >> 3);
                const int64_t row = i < w.rows ? row_at(w, i) - top : 0;
                bo[a][d] = i < w.rows ? (uint32_t)(row * p.base_stride + 8 * (l & 7)) * os : ring::kOOB;
                oo[a][d] = i < w.rows ? (uint32_t)(row * p.out_stride + 8 * (l & 7)) * os : ring::kOOB;
            }
        auto fetch = [&](Line8<O> (&o)[MT][2], int c) {
            const bool in = c + 8 * (l & 7) < col1;
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int d = 0; d < 2; ++d) o[a][d].load(rb, in && bo[a][d] != ring::kOOB ? bo[a][d] + (uint32_t)c * os : ring::kOOB);
        };
        auto weights = [&](i32x4 (&v)[WL], int c) {   // columns past n: 0
#pragma unroll
            for (int u = 0; u < WL; ++u)
                v[u] = __builtin_amdgcn_raw_buffer_load_b128(rw, at[u] >= 0 ? (uint32_t)c * p.r * 2u + 16u * (t + NT * u) : ring::kOOB, 0, 0);
        };
        auto put = [&](const i32x4 (&v)[WL], int slot) {
#pragma unroll
            for (int u = 0; u < WL; ++u)
                if (at[u] >= 0) *(i32x4*)(sm.s.w[slot] + at[u]) = v[u];
        };
        i32x4 wv[WL];
        Line8<O> o[MT][2], next[MT][2];
        weights(wv, col0);
        fetch(o, col0);
        __syncthreads();                    // the zeros are written
        put(wv, 0);
        weights(wv, col0 + 64);
        int slot = 0;
        for (int c = col0; c < col1; c += 64, slot ^= 1) {
            __syncthreads();                // this step's weights are in LDS, and the last one's have been read
            fetch(next, c + 64);
            f32x4 acc[MT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf16x8 m[STEPS];
#pragma unroll
                for (int s = 0; s < STEPS; ++s) m[s] = slot_frag(sm.s.w[slot], 16 * j + i16, s);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    acc[a][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < STEPS; ++s)
#pragma unroll
                        for (int z = 0; z < 2; ++z) acc[a][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(m[s], x[a][s][z], acc[a][j], 0, 0, 0);
                }
            }
            float* strip = sm.s.strips[wave];
            const bool in = c + 8 * (l & 7) < col1;
#pragma unroll
            for (int a = 0; a < MT; ++a) {
#pragma unroll
                for (int j = 0; j < 4; ++j) *(f32x4*)(strip + i16 * SP + 16 * j + 4 * q) = acc[a][j];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const float* from = strip + (8 * d + (l >> 3)) * SP + 8 * (l & 7);
                    const f32x4 lo = *(const f32x4*)from, hi = *(const f32x4*)(from + 4);
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) { v[e] = lo[e] + o[a][d].get(e); v[4 + e] = hi[e] + o[a][d].get(4 + e); }
                    Line8<O>::store(ro, in && oo[a][d] != ring::kOOB ? oo[a][d] + (uint32_t)c * os : ring::kOOB, v);
                }
            }
            put(wv, slot ^ 1);
            weights(wv, c + 128);
#pragma unroll
            for (int a = 0; a < MT; ++a) { o[a][0] = next[a][0]; o[a][1] = next[a][1]; }
        }
    }
}

// ---------------------------------------------------------------------------------------------------------------
// turn: two of [g, rows, cols] -> [g, cols, rows], in tiles of 4096 values as wide as the narrower side wants

struct Turn { const void* a; void* at; int rows, cols, lg, tr, tc; };   // 2^lg columns a tile, tr x tc tiles
template <typename T>
__global__ __launch_bounds__(NT) void turn(Turn p0, Turn p1, int first) {   // the first `first` workgroups: p0
    __shared__ T s[4096 + 2048];
    const bool one = (int)blockIdx.x >= first;
    const Turn& p = one ? p1 : p0;
    const int id = one ? blockIdx.x - first : blockIdx.x;
    const int w = 1 << p.lg, hgt = 4096 >> p.lg, pitch = w + (w < 64 ? 2 : 8);
    const int c0 = w * (id % p.tc), r0 = hgt * ((id / p.tc) % p.tr);
    const int64_t off = (int64_t)(id / p.tc / p.tr) * p.rows * p.cols;
    const T* a = (const T*)p.a + off;
    T* at = (T*)p.at + off;
    T v[4096 / NT];   // all of a thread's loads in flight
#pragma unroll
    for (int u = 0; u < 4096 / NT; ++u) {
        const int e = threadIdx.x + NT * u, r = min(r0 + (e >> p.lg), p.rows - 1), c = min(c0 + (e & (w - 1)), p.cols - 1);
        v[u] = a[(int64_t)r * p.cols + c];
    }
#pragma unroll
    for (int u = 0; u < 4096 / NT; ++u) {
        const int e = threadIdx.x + NT * u;
        s[(e >> p.lg) * pitch + (e & (w - 1))] = v[u];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4096 / NT; ++u) {
        const int e = threadIdx.x + NT * u, c = e >> (12 - p.lg), r = e & (hgt - 1);
        if (r0 + r < p.rows && c0 + c < p.cols) at[(int64_t)(c0 + c) * p.rows + r0 + r] = s[r * pitch + c];
    }
}

// ---------------------------------------------------------------------------------------------------------------
// outer: sums over rows.  A workgroup takes a chunk of rows of one group and TC columns of x (then da [r, k]) or of
// dout (then db [n, r]), some rows at a time through LDS.  The narrow operand (u or v) is the first, so a lane ends with four consecutive j
// of one column.

// What a wave holds of da's or db's sums over one chunk (NB x CB blocks, lane: four consecutive j of one column) to its place.
struct Chunk { int h, part, first, rows, c0, cols; bool of_x, whole; };
template <int NB, int CB>
__device__ inline void outer_store(const Outer& p, const Chunk& w, const f32x4 (&acc)[NB][CB]) {
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, q = l >> 4, i16 = l & 15;
    // one chunk: the result; more: the chunk's part, at a place that no other chunk of such a group has (two such
    // chunks begin in the same `chunk` rows only if one is a group's first and the other is not)
    const float scale = w.whole && p.scaling ? p.scaling[w.h] : 1.f;
    const int64_t per = (int64_t)(p.k + p.n) * p.r;
    float* part_at = p.parts + (2 * (int64_t)(w.first / p.chunk) + (w.part == 0)) * per;
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            const int col = w.c0 + 16 * (CB * wave + c) + i16;
            if (col >= w.cols) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 16 * a + 4 * q + e;
                if (j >= p.r) continue;
                const int64_t at = w.of_x ? (int64_t)j * p.k + col : (int64_t)col * p.r + j;
                if (!w.whole) part_at[(w.of_x ? 0 : (int64_t)p.k * p.r) + at] = acc[a][c][e];
                else {
                    const float v = acc[a][c][e] * scale;
                    const int64_t to = (int64_t)w.h * (w.of_x ? p.k : p.n) * p.r + at;
                    void* dst = w.of_x ? p.da : p.db;
                    if (p.grads_bf16) Out8<uint16_t>::put((uint16_t*)dst + to, v);
                    else ((float*)dst)[to] = v;
                }
            }
        }
}
// Which chunk of which group, and which columns (TC of them) a workgroup has; false: none (a group without rows is cleared).
template <int TC>
__device__ inline bool outer_chunk(const Outer& p, Tables& tab, Chunk& w) {
    int tiles, covered;
    build_tables<NT>(p.group_sizes, p.g, p.m, p.chunk, 1, tab, &tiles, &covered);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = tab.flags;
    const int xt = (p.k + TC - 1) / TC, dt = (p.n + TC - 1) / TC;
    const int place = blockIdx.x / (xt + dt), id = tiles - 1 - place, ct = blockIdx.x - place * (xt + dt);   // from the end
    if (id < 0) {
        // With no more rows than a chunk every group with rows has one, join is not launched, and the places left over are
        // the groups' without rows: h - tile_off[h] of them lie before group h.
        const int e = -1 - id;
        if (p.m > p.chunk || e >= p.g - tiles) return false;
        int lo = 0, hi = p.g - 1;   // the first h with more than e such groups up to it
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (mid + 1 - tab.tile_off[mid + 1] > e) hi = mid; else lo = mid + 1;
        }
        const bool in_x = ct < xt;
        const int from = (in_x ? ct : ct - xt) * TC, width = min(TC, (in_x ? p.k : p.n) - from);
        for (int i = threadIdx.x; i < width * p.r; i += NT) {
            const int64_t at = in_x ? (int64_t)lo * p.r * p.k + (int64_t)(i / width) * p.k + from + i % width
                                    : (int64_t)lo * p.n * p.r + (int64_t)from * p.r + i;
            void* dst = in_x ? p.da : p.db;
            if (p.grads_bf16) ((uint16_t*)dst)[at] = 0;
            else ((float*)dst)[at] = 0.f;
        }
        return false;
    }
    w.h = find_group(tab.tile_off, p.g, id);
    w.part = id - tab.tile_off[w.h];
    const int size = tab.row_off[w.h + 1] - tab.row_off[w.h];
    w.first = tab.row_off[w.h] + w.part * p.chunk;
    w.rows = min(p.chunk, size - w.part * p.chunk);
    w.whole = size <= p.chunk;
    w.of_x = ct < xt;
    w.c0 = (w.of_x ? ct : ct - xt) * TC;
    w.cols = w.of_x ? p.k : p.n;
    return true;
}

// bf16 dout, and x in bf16 or e4m3.  The wide operand's rows lie in LDS as [BR][256], 32-byte units XOR'ed with the row so
// that the eight rows which half of a transposing read's lanes touch lie in distinct banks; u or v lies there turned,
// [part][j][row], so that a fragment is one read.  A thread holds the next BR rows' part while these are multiplied.
template <bool X8, int NB, int P, int CB>   // X8: x is e4m3; CB: 16-column blocks a wave
__global__ __launch_bounds__(NT) void outer16(Outer p) {
    constexpr int BR = NB <= 4 ? 64 : 32, TC = 64 * CB, NP = BR + 8;
    constexpr int RG = BR / 4, JB = NT / (16 * RG), PASSES = (NB + JB - 1) / JB;   // narrow: four rows of a j a thread and pass
    __shared__ union {
        Tables tab;
        struct {
            __attribute__((aligned(16))) uint16_t wide[BR * 256];
            __attribute__((aligned(16))) uint16_t nar[P][16 * NB * NP];
        };
    } sm;
    Chunk w;
    if (!outer_chunk<TC>(p, sm.tab, w)) return;
    __syncthreads();   // the tables' memory is used again
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;
    const int c1 = min(w.cols, w.c0 + TC);
    f32x4 acc[NB][CB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < CB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto unit = [](int row, int col) { return row * 256 + ((((col >> 4) ^ ((row & 3) | (((row >> 3) & 1) << 2))) << 4) | (col & 15)); };

    // the narrow operand: j = 16 (JB pass + ...) + t % 16, rows 4 (t / 16 % RG) .. + 3
    const int nj = 16 * (t / (16 * RG)) + (t & 15), nr = 4 * ((t >> 4) % RG);
    const float* nsrc = (w.of_x ? p.u : p.v) + (int64_t)(w.first + nr) * p.r + nj;
    float nv[PASSES][4];
    auto load_nar = [&](int r0) {
#pragma unroll
        for (int z = 0; z < PASSES; ++z)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                nv[z][e] = nj + 16 * JB * z < p.r && r0 + nr + e < w.rows ? nsrc[(int64_t)(r0 + e) * p.r + 16 * JB * z] : 0.f;
    };
    auto store_nar = [&]() {
#pragma unroll
        for (int z = 0; z < PASSES; ++z) {
            if (NB < JB && nj >= 16 * NB) continue;
            uint16_t s[4][P];
#pragma unroll
            for (int e = 0; e < 4; ++e) split<P>(nv[z][e], s[e]);
#pragma unroll
            for (int i = 0; i < P; ++i)
                *(i32x2*)(&sm.nar[i][(nj + 16 * JB * z) * NP + nr]) = i32x2{s[0][i] | s[1][i] << 16, s[2][i] | s[3][i] << 16};
        }
    };
    auto multiply = [&]() {
#pragma unroll
        for (int s = 0; s < BR / 32; ++s) {
            bf16x8 b[CB];
#pragma unroll
            for (int c = 0; c < CB; ++c) {   // rows 32 s + 8 q .. + 7 of one column, from two transposing reads of 4 x 16 values
                const int row = 32 * s + 8 * q + (i16 >> 2), col = 16 * (CB * wave + c) + 4 * (i16 & 3);
                const i16x4 lo = lds_read_tr16(sm.wide + unit(row, col)), hi = lds_read_tr16(sm.wide + unit(row + 4, col));
                typedef short i16x8 __attribute__((ext_vector_type(8)));
                const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                b[c] = __builtin_bit_cast(bf16x8, v);
            }
#pragma unroll
            for (int a = 0; a < NB; ++a)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const bf16x8 n = *(const bf16x8*)(&sm.nar[i][(16 * a + i16) * NP + 32 * s + 8 * q]);
#pragma unroll
                    for (int c = 0; c < CB; ++c) acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n, b[c], acc[a][c], 0, 0, 0);
                }
        }
    };
    auto steps = [&](auto& load, auto& store) {
        load(0);
        load_nar(0);
        for (int r0 = 0; r0 < w.rows; r0 += BR) {
            store();
            store_nar();
            __syncthreads();
            if (r0 + BR < w.rows) {
                load(r0 + BR);
                load_nar(r0 + BR);
            }
            multiply();
            __syncthreads();
        }
    };
    if (X8 && w.of_x) {   // row t / (256 / BR'), blocks of 32 columns
        constexpr int BLK = BR / 32, TR = 8 / BLK;              // blocks a thread, threads a row
        const int row = t / TR, col = 32 * BLK * (t % TR), c = w.c0 + col;
        const uint8_t* src = (const uint8_t*)p.x + (int64_t)(w.first + row) * p.k + c;
        const uint8_t* scl = p.x_scale + (int64_t)(w.first + row) * (p.k >> 5) + (c >> 5);
        i32x4 v[BLK][2];
        int byte[BLK];
        auto load = [&](int r0) {
#pragma unroll
            for (int b = 0; b < BLK; ++b) {
                v[b][0] = v[b][1] = i32x4{0, 0, 0, 0};
                byte[b] = 0;
                if (r0 + row < w.rows && c + 32 * b < c1) {
                    const i32x4* at = (const i32x4*)(src + (int64_t)r0 * p.k + 32 * b);
                    v[b][0] = at[0];
                    v[b][1] = at[1];
                    byte[b] = scl[(int64_t)r0 * (p.k >> 5) + b];
                }
            }
        };
        auto store = [&]() {
#pragma unroll
            for (int b = 0; b < BLK; ++b) {
                const float s = __uint_as_float((uint32_t)byte[b] << 23);   // exponent field 255 is NaN to the conversion
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    i32x4 o;
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        const uint32_t x = (uint32_t)v[b][i >> 1][2 * (i & 1) + d];
                        o[2 * d] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, false));
                        o[2 * d + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, true));
                    }
                    *(i32x4*)(sm.wide + unit(row, col + 32 * b + 8 * i)) = o;
                }
            }
        };
        steps(load, store);
    } else {   // rows t / 32 + 8 i, eight columns
        const int row = t >> 5, col = 8 * (t & 31), c = w.c0 + col;
        const int64_t stride = w.of_x ? p.k : p.n;
        const uint16_t* src = (const uint16_t*)(w.of_x ? p.x : p.dout) + (int64_t)(w.first + row) * stride + c;
        i32x4 v[BR / 8];
        const uint16_t* end = (const uint16_t*)(w.of_x ? p.x : p.dout) + (int64_t)p.m * stride;
        i32x4 mask;
#pragma unroll
        for (int d = 0; d < 4; ++d) mask[d] = c + 2 * d + 2 <= c1 ? -1 : c + 2 * d + 1 == c1 ? 0xffff : 0;
        auto load = [&](int r0) {
#pragma unroll
            for (int i = 0; i < BR / 8; ++i) {
                v[i] = i32x4{0, 0, 0, 0};
                if (r0 + row + 8 * i >= w.rows || c >= c1) continue;
                const uint16_t* at = src + (int64_t)(r0 + 8 * i) * stride;
                if (at + 8 <= end) v[i] = *(const i32x4_any*)at;   // what lies behind the row is masked later, so that no load waits
                else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < c1) v[i][e >> 1] |= (int)((uint32_t)at[e] << (16 * (e & 1)));
                }
            }
        };
        auto store = [&]() {
#pragma unroll
            for (int i = 0; i < BR / 8; ++i) *(i32x4*)(sm.wide + unit(row + 8 * i, col)) = v[i] & mask;
        };
        steps(load, store);
    }
    outer_store<NB, CB>(p, w, acc);
}

// fp32: both operands are read from LDS as they lie, instruction i of 32 rows taking rows 4 i + q.
constexpr int WP32 = 256 + 4;
template <int NB, int CB>
__global__ __launch_bounds__(NT) void outer32(Outer p) {
    constexpr int TC = 64 * CB, NP = 16 * NB + 4, NPER = 32 * 16 * NB / NT;
    __shared__ Tables tab;
    __shared__ __attribute__((aligned(16))) float wide[32 * WP32];
    __shared__ __attribute__((aligned(16))) float nar[32 * NP];
    Chunk w;
    if (!outer_chunk<TC>(p, tab, w)) return;
    const float* nsrc = w.of_x ? p.u : p.v;
    const float* wsrc = (const float*)(w.of_x ? p.x : p.dout);
    const int t = threadIdx.x, l = t & 63, wave = t >> 6, q = l >> 4, i16 = l & 15;
    const int c = w.c0 + 8 * (t & 31), c1 = min(w.cols, w.c0 + TC);
    f32x4 acc[NB][CB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < CB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 v[4][2];      // row t / 32 + 8 i, eight columns
    float nv[NPER];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + (t >> 5) + 8 * i;
            v[i][0] = v[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (r >= w.rows || c >= c1) continue;
            const float* at = wsrc + (int64_t)(w.first + r) * w.cols + c;
            if (at + 8 <= wsrc + (int64_t)p.m * w.cols) {   // what lies behind the row is masked later, so that no load waits
                v[i][0] = *(const f32x4_any*)at;
                v[i][1] = *(const f32x4_any*)(at + 4);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < c1) v[i][e >> 2][e & 3] = at[e];
            }
        }
#pragma unroll
        for (int e = 0; e < NPER; ++e) {
            const int at = t + NT * e, i = at / (16 * NB), j = at % (16 * NB);
            nv[e] = r0 + i < w.rows && j < p.r ? nsrc[(int64_t)(w.first + r0 + i) * p.r + j] : 0.f;
        }
    };
    auto store = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float* at = wide + ((t >> 5) + 8 * i) * WP32 + 8 * (t & 31);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e >= c1) v[i][e >> 2][e & 3] = 0.f;
            *(f32x4*)at = v[i][0];
            *(f32x4*)(at + 4) = v[i][1];
        }
#pragma unroll
        for (int e = 0; e < NPER; ++e) {
            const int at = t + NT * e;
            nar[at / (16 * NB) * NP + at % (16 * NB)] = nv[e];
        }
    };
    load(0);
    for (int r0 = 0; r0 < w.rows; r0 += 32) {
        store();
        __syncthreads();
        if (r0 + 32 < w.rows) load(r0 + 32);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            float b[CB];
#pragma unroll
            for (int c = 0; c < CB; ++c) b[c] = wide[(4 * s + q) * WP32 + 16 * (CB * wave + c) + i16];
#pragma unroll
            for (int a = 0; a < NB; ++a) {
                const float n = nar[(4 * s + q) * NP + 16 * a + i16];
#pragma unroll
                for (int c = 0; c < CB; ++c) acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(n, b[c], acc[a][c], 0, 0, 0);
            }
        }
        __syncthreads();
    }
    outer_store<NB, CB>(p, w, acc);
}

// join: groups of several chunks, in their order; groups without rows are 0.  V consecutive values a thread.
template <int V>
__global__ __launch_bounds__(NT) void join(Outer p, int blocks) {
    __shared__ Tables tab;
    const int h = blockIdx.x / blocks, b = blockIdx.x - h * blocks;
    int first = 0, rows = 0;
    if (p.g <= 64) {   // as in sorted_tile
        const int l = threadIdx.x & 63;
        uint32_t end = l < p.g ? (uint32_t)min(max(p.group_sizes[l], 0), p.m) : 0u;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t u = (uint32_t)__shfl_up((int)end, d, 64);
            if (l >= d) end = min(end + u, (uint32_t)p.m);
        }
        first = h ? __shfl((int)end, h - 1, 64) : 0;
        rows = __shfl((int)end, h, 64) - first;
    } else {
        int tiles, covered;
        build_tables<NT>(p.group_sizes, p.g, p.m, p.chunk, 1, tab, &tiles, &covered);
        first = tab.row_off[h];
        rows = tab.row_off[h + 1] - first;
    }
    if (rows > 0 && rows <= p.chunk) return;
    const int chunks = (rows + p.chunk - 1) / p.chunk;
    const float scale = p.scaling ? p.scaling[h] : 1.f;
    const int64_t ka = (int64_t)p.k * p.r, per = (int64_t)(p.k + p.n) * p.r;
    for (int64_t e = ((int64_t)b * NT + threadIdx.x) * V; e < per; e += (int64_t)blocks * NT * V) {
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = 0.f;
        for (int c = 0; c < chunks; c += 4) {   // four chunks' loads at a time, added in order
            float f[4][V];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int at = c + u;
                const float* from = p.parts + (2 * (int64_t)((first + min(at, chunks - 1) * p.chunk) / p.chunk) + (at == 0)) * per + e;
                if constexpr (V == 4) {
                    const f32x4 q = at < chunks ? *(const f32x4_any*)from : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < V; ++i) f[u][i] = q[i];
                } else {
                    f[u][0] = at < chunks ? *from : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] += f[u][i];
        }
        void* dst = e < ka ? p.da : p.db;
        const int64_t to = e < ka ? h * ka + e : (int64_t)h * p.n * p.r + (e - ka);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = rows > 0 ? s[i] * scale : 0.f;
            if (p.grads_bf16) Out8<uint16_t>::put((uint16_t*)dst + to + i, v);
            else ((float*)dst)[to + i] = v;
        }
    }
}

}  // namespace lora

// ---------------------------------------------------------------------------------------------------------------
// launches

static int64_t up64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Parts of the long axis: about a thousand workgroups, no part shorter than one piece of each wave, and for many rows
// parts whose sums are few beside the rows themselves.
int lora_splits(int64_t m, int64_t k, int r, int g) {
    const int64_t tiles = std::max<int64_t>(1, up64(m, 64)), few = std::min<int64_t>(m, g);
    const int64_t pieces = up64(k, 4 * lora::KC), want = few > tiles ? 512 / few : 1024 / tiles;
    const int64_t most = m >= 1024 ? std::min<int64_t>(8, k / (16 * r)) : 32;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(most, want), pieces));
}
// Rows that a workgroup of the row sums takes: about 1024 workgroups, and chunks long enough that their parts are few.
int lora_chunk(int64_t m, int64_t k, int64_t n) {
    const int64_t tiles = up64(k, 256) + up64(n, 256);
    const int64_t c = up64(up64(m * tiles, 1024), 32) * 32;
    return (int)std::min<int64_t>(2048, std::max<int64_t>(512, c));
}

// Whether an adapter has enough rows on average to fill tiles of more than 16
static bool lora_many(const lora::Rows& r) {
    return (r.group_sizes ? r.m / r.g : std::min<int64_t>(r.m, r.chunk) / std::max(1, r.slots)) >= 32;
}
void lora_rows(lora::Rows& r) {
    r.chunk = (int)std::min<int64_t>(lora::MAXCHUNK, std::max<int64_t>(256, up64((int64_t)32 * r.g, 256) * 256));
    r.slots = (int)std::min<int64_t>(r.g, std::min<int64_t>(r.m, r.chunk));
}
static int64_t lora_tiles(const lora::Rows& r, int tm) {
    return r.group_sizes ? up64(r.m, tm) + r.g + 1 : std::max<int64_t>(1, up64(r.m, r.chunk)) * (r.slots + r.chunk / lora::NONE);
}
static int lora_nb(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : r <= 128 ? 8 : 16; }

// Whether every launch over these rows and columns of the second product stays below a launch's workgroups: a call is
// refused before the first of its launches or not at all.
bool lora_grid_ok(const lora::Rows& r, int64_t n) { return lora_tiles(r, 16) * std::max<int64_t>(1, up64(n, 2048)) <= kMaxBlocks; }
// the same for what the gradients add: both weights turned, and the row sums over 64 columns at the narrowest
bool lora_grad_grid_ok(int64_t m, int64_t k, int64_t n, int g) {
    const int64_t sums = (up64(m, lora_chunk(m, k, n)) + g) * (up64(k, 64) + up64(n, 64));
    return sums <= kMaxBlocks && g * (up64(k, 16) + up64(n, 16)) <= kMaxBlocks;
}

template <typename T, int NB>
static hipError_t shrink_t(const lora::Shrink& p, hipStream_t s) {
    constexpr int U = NB == 1 ? 4 : NB <= 4 ? 2 : 1;
    const int64_t tiles = lora_tiles(p.rows, 16);
    if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((lora::shrink<T, NB, U>), dim3((uint32_t)tiles, p.splits), dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
template <typename T, int NB>
static hipError_t shrink_staged_t(const lora::Shrink& p, hipStream_t s) {
    const int64_t tiles = lora_tiles(p.rows, 64);
    if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((lora::shrink_staged<T, NB>), dim3((uint32_t)tiles, p.splits), dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
template <typename T, int NB, int TEAM, int D>
static hipError_t shrink_ring_t(const lora::Shrink& p, hipStream_t s) {
    const int64_t tiles = lora_tiles(p.rows, 16 * TEAM);
    if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((lora::shrink_ring<T, NB, TEAM, D>), dim3((uint32_t)tiles, p.splits), dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
static bool shrink_lines(const lora::Shrink& p, int64_t es) {   // rows of whole 16 bytes
    return (uintptr_t)p.x % 16 == 0 && (uintptr_t)p.w % 16 == 0 && p.stride * es % 16 == 0 && p.k * es % 16 == 0;
}
template <typename T>
static hipError_t shrink_nb(const lora::Shrink& p, hipStream_t s) {
    const int nb = lora_nb(p.r);
    const bool many = lora_many(p.rows);
    if (shrink_lines(p, sizeof(T))) {
        switch (nb) {
            case 1: return many ? shrink_ring_t<T, 1, 4, 5>(p, s) : shrink_ring_t<T, 1, 1, 4>(p, s);
            case 2: return many ? shrink_ring_t<T, 2, 4, 5>(p, s) : shrink_ring_t<T, 2, 1, 3>(p, s);
            case 4: return many ? shrink_ring_t<T, 4, 4, 4>(p, s) : shrink_ring_t<T, 4, 1, 3>(p, s);
            case 8: return many ? shrink_ring_t<T, 8, 4, 3>(p, s) : shrink_ring_t<T, 8, 1, 2>(p, s);
            default: return shrink_ring_t<T, 16, 4, 3>(p, s);   // a ring a wave would not fit the LDS
        }
    }
    if (many) {
        switch (nb) {
            case 1: return shrink_staged_t<T, 1>(p, s);
            case 2: return shrink_staged_t<T, 2>(p, s);
            case 4: return shrink_staged_t<T, 4>(p, s);
            case 8: return shrink_staged_t<T, 8>(p, s);
            default: return shrink_staged_t<T, 16>(p, s);
        }
    }
    switch (nb) {
        case 1: return shrink_t<T, 1>(p, s);
        case 2: return shrink_t<T, 2>(p, s);
        case 4: return shrink_t<T, 4>(p, s);
        case 8: return shrink_t<T, 8>(p, s);
        default: return shrink_t<T, 16>(p, s);
    }
}
hipError_t launch_lora_shrink(const lora::Shrink& p, bool bf16, hipStream_t s) {
    return bf16 ? shrink_nb<uint16_t>(p, s) : shrink_nb<float>(p, s);
}

template <typename T, typename O, int NB, int MT>
static hipError_t expand_t(lora::Expand p, hipStream_t s) {
    const int64_t tiles = lora_tiles(p.rows, 16 * MT);
    p.cols = 2048;
    while (p.cols > 256 && tiles * up64(p.n, p.cols) < 1024) p.cols /= 2;
    p.col_tiles = (int)std::max<int64_t>(1, up64(p.n, p.cols));
    if (tiles * p.col_tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)(tiles * p.col_tiles));
    if (p.r % 8 == 0) hipLaunchKernelGGL((lora::expand<T, O, NB, MT, true>), grid, dim3(lora::NT), 0, s, p);
    else hipLaunchKernelGGL((lora::expand<T, O, NB, MT, false>), grid, dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
template <typename O, int NB, int MT>
static hipError_t expand_lines_t(lora::Expand p, hipStream_t s) {
    const int64_t tiles = lora_tiles(p.rows, 64 * MT);
    p.cols = 2048;
    while (p.cols > 256 && tiles * up64(p.n, p.cols) < 1024) p.cols /= 2;
    p.col_tiles = (int)std::max<int64_t>(1, up64(p.n, p.cols));
    if (tiles * p.col_tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((lora::expand_lines<O, NB, MT>), dim3((uint32_t)(tiles * p.col_tiles)), dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
// expand_lines: 16-byte rows and ranks, and 32-bit offsets over an adapter's weights and over the rows of a tile (of a
// chunk, in any order)
template <typename O> static bool expand_lines_ok(const lora::Expand& p) {
    const int64_t span = (p.rows.group_sizes ? 256 : lora::MAXCHUNK) * (int64_t)sizeof(O);
    return p.r % 8 == 0 && p.n % 8 == 0 && p.base_stride * sizeof(O) % 16 == 0 && p.out_stride * sizeof(O) % 16 == 0 &&
           (uintptr_t)p.base % 16 == 0 && (uintptr_t)p.out % 16 == 0 && (uintptr_t)p.w % 16 == 0 &&
           ((int64_t)p.n + 256) * p.r * 2 < (int64_t(1) << 31) && std::max(p.base_stride, p.out_stride) * span < (int64_t(1) << 31);
}
template <typename T, typename O>
static hipError_t expand_nb(const lora::Expand& p, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (lora_many(p.rows) && expand_lines_ok<O>(p)) {
            switch (lora_nb(p.r)) {
                case 1: return expand_lines_t<O, 1, 2>(p, s);
                case 2: return expand_lines_t<O, 2, 2>(p, s);
                case 4: return expand_lines_t<O, 4, 2>(p, s);
                case 8: return expand_lines_t<O, 8, 1>(p, s);
                default: return expand_lines_t<O, 16, 1>(p, s);
            }
        }
    }
    // few rows and columns: small tiles (more workgroups, and half the instructions for each to fetch)
    const bool many = up64(p.rows.m, 64) * up64(p.n, 256) >= 512 && lora_many(p.rows);
    switch (lora_nb(p.r)) {
        case 1: return many ? expand_t<T, O, 1, 2>(p, s) : expand_t<T, O, 1, 1>(p, s);
        case 2: return many ? expand_t<T, O, 2, 2>(p, s) : expand_t<T, O, 2, 1>(p, s);
        case 4: return many ? expand_t<T, O, 4, 2>(p, s) : expand_t<T, O, 4, 1>(p, s);
        case 8: return many ? expand_t<T, O, 8, 2>(p, s) : expand_t<T, O, 8, 1>(p, s);
        default: return expand_t<T, O, 16, 1>(p, s);
    }
}
// Few rows an adapter, rows of whole 16 bytes, and first weights of at most 128 KiB an adapter: both products in one launch.
// (One token at rank 16 and 4096 columns: 7.7 us in one launch, 4.1 + 5.2 in two, and the host's 2.8 for the second; 96 rows at 64
// adapters of 448 KiB: 20 us in one, since every workgroup streams the weights for itself, 7.8 + 6.0 in two.)
bool lora_both_ok(const lora::Shrink& p, bool bf16) {
    const int64_t es = bf16 ? 2 : 4;
    return !lora_many(p.rows) && p.r <= 64 && p.r * (int64_t)p.k * es <= (1 << 17) && shrink_lines(p, es);
}
template <typename T, typename O, int NB, int D>
static hipError_t both_t(const lora::Shrink& sh, lora::Expand p, hipStream_t s) {
    const int64_t tiles = lora_tiles(p.rows, 16);
    p.cols = 4096;
    // about a workgroup a compute unit, as each contracts the rows again (64 rows of 64 adapters of rank 16, k = n = 4096:
    // 11.4 us, with 512 workgroups 14, with 1024 18)
    while (p.cols > 256 && tiles * up64(p.n, p.cols) < 256) p.cols /= 2;
    p.col_tiles = (int)std::max<int64_t>(1, up64(p.n, p.cols));
    if (tiles * p.col_tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)(tiles * p.col_tiles));
    if (p.r % 8 == 0) hipLaunchKernelGGL((lora::both<T, O, NB, D, true>), grid, dim3(lora::NT), 0, s, lora::Both{sh, p});
    else hipLaunchKernelGGL((lora::both<T, O, NB, D, false>), grid, dim3(lora::NT), 0, s, lora::Both{sh, p});
    return hipGetLastError();
}
template <typename T, typename O>
static hipError_t both_nb(const lora::Shrink& sh, const lora::Expand& p, hipStream_t s) {
    switch (lora_nb(p.r)) {
        case 1: return both_t<T, O, 1, 4>(sh, p, s);
        case 2: return both_t<T, O, 2, 3>(sh, p, s);
        default: return both_t<T, O, 4, 3>(sh, p, s);
    }
}
hipError_t launch_lora_both(const lora::Shrink& sh, const lora::Expand& p, bool bf16, bool out_bf16, hipStream_t s) {
    if (bf16) return out_bf16 ? both_nb<uint16_t, uint16_t>(sh, p, s) : both_nb<uint16_t, float>(sh, p, s);
    return out_bf16 ? both_nb<float, uint16_t>(sh, p, s) : both_nb<float, float>(sh, p, s);
}
hipError_t launch_lora_expand(const lora::Expand& p, bool bf16, bool out_bf16, hipStream_t s) {
    if (bf16) return out_bf16 ? expand_nb<uint16_t, uint16_t>(p, s) : expand_nb<uint16_t, float>(p, s);
    return out_bf16 ? expand_nb<float, uint16_t>(p, s) : expand_nb<float, float>(p, s);
}

static lora::Turn turn_of(const void* a, void* at, int rows, int cols) {
    int lg = 4;
    while (lg < 8 && (1 << lg) < cols && (4096 >> lg) > rows) ++lg;
    while (lg < 6 && (1 << lg) < cols) ++lg;
    return {a, at, rows, cols, lg, (int)up64(rows, 4096 >> lg), (int)up64(cols, 1 << lg)};
}
hipError_t launch_lora_turn(const void* a, void* at, int rows, int cols, const void* b, void* bt, int rows_b, int cols_b, bool bf16, int g,
                            hipStream_t s) {
    const lora::Turn p = turn_of(a, at, rows, cols), q = turn_of(b, bt, rows_b, cols_b);
    const int64_t first = a ? (int64_t)p.tr * p.tc * g : 0, blocks = first + (b ? (int64_t)q.tr * q.tc * g : 0);
    if (blocks == 0) return hipSuccess;
    if (blocks > kMaxBlocks) return hipErrorInvalidConfiguration;
    if (bf16) hipLaunchKernelGGL(lora::turn<uint16_t>, dim3((uint32_t)blocks), dim3(lora::NT), 0, s, p, q, (int)first);
    else hipLaunchKernelGGL(lora::turn<float>, dim3((uint32_t)blocks), dim3(lora::NT), 0, s, p, q, (int)first);
    return hipGetLastError();
}

enum class OuterX { bf16, e4m3, f32 };
template <OuterX X, int NB, int P, int CB>
static hipError_t outer_t(const lora::Outer& p, hipStream_t s) {
    const int64_t tiles = up64(p.m, p.chunk) + p.g, cols = up64(p.k, 64 * CB) + up64(p.n, 64 * CB);
    if (tiles * cols > kMaxBlocks) return hipErrorInvalidConfiguration;
    if (tiles * cols == 0) return hipSuccess;
    const dim3 grid((uint32_t)(tiles * cols));
    if constexpr (X == OuterX::f32) hipLaunchKernelGGL((lora::outer32<NB, CB>), grid, dim3(lora::NT), 0, s, p);
    else hipLaunchKernelGGL((lora::outer16<X == OuterX::e4m3, NB, P, CB>), grid, dim3(lora::NT), 0, s, p);
    return hipGetLastError();
}
template <OuterX X, int P>
static hipError_t outer_nb(const lora::Outer& p, hipStream_t s) {
    // Few workgroups: narrower ones (375 fp32 rows of 5 groups, k 1030, n 515: 15 us with wide ones, 11 with these; 109 bf16
    // rows over 64 groups, k 4081, n 384: 11 with wide ones, 25 with these).  Every row may be another group's.
    const int64_t groups = std::max<int64_t>(up64(p.m, p.chunk), std::min<int64_t>(p.g, p.m));
    if (p.r <= 64 && groups * (up64(p.k, 256) + up64(p.n, 256)) < 256) {
        switch (lora_nb(p.r)) {
            case 1: return outer_t<X, 1, P, 1>(p, s);
            case 2: return outer_t<X, 2, P, 1>(p, s);
            default: return outer_t<X, 4, P, 1>(p, s);
        }
    }
    switch (lora_nb(p.r)) {
        case 1: return outer_t<X, 1, P, 4>(p, s);
        case 2: return outer_t<X, 2, P, 4>(p, s);
        case 4: return outer_t<X, 4, P, 4>(p, s);
        case 8: return outer_t<X, 8, P, 2>(p, s);
        default: return outer_t<X, 16, P, 1>(p, s);
    }
}
hipError_t launch_lora_outer(const lora::Outer& p, bool bf16, hipStream_t s) {
    hipError_t e;
    if (!bf16) e = outer_nb<OuterX::f32, 1>(p, s);
    else if (p.x_scale) e = p.grads_bf16 ? outer_nb<OuterX::e4m3, 2>(p, s) : outer_nb<OuterX::e4m3, 3>(p, s);
    else e = p.grads_bf16 ? outer_nb<OuterX::bf16, 2>(p, s) : outer_nb<OuterX::bf16, 3>(p, s);
    if (e != hipSuccess) return e;
    const int64_t per = (int64_t)(p.k + p.n) * p.r;
    if (per == 0 || p.m <= p.chunk) return hipSuccess;   // no group has two chunks
    const bool four = (int64_t)p.k * p.r % 4 == 0 && (int64_t)p.n * p.r % 4 == 0;   // neither matrix ends inside a thread's values
    const int blocks = (int)std::min<int64_t>(up64(per, lora::NT * (four ? 4 : 1)), std::max<int64_t>(1, 4096 / p.g));
    if ((int64_t)blocks * p.g > kMaxBlocks) return hipErrorInvalidConfiguration;
    if (four) hipLaunchKernelGGL(lora::join<4>, dim3((uint32_t)(blocks * p.g)), dim3(lora::NT), 0, s, p, blocks);
    else hipLaunchKernelGGL(lora::join<1>, dim3((uint32_t)(blocks * p.g)), dim3(lora::NT), 0, s, p, blocks);
    return hipGetLastError();
}

}  // namespace gg
