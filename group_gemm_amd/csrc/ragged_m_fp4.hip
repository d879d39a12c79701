// ragged_m_fp4.hip -- the MXFP4 non-contracting ragged dot on gfx950: out[r, :] = lhs[r, :] . rhs[h]^T for
// the rows r of group h, both operands e2m1 codes with k contiguous and E8M0 scales in panels
// [ceil(k/256), rows, 8], fp32 accumulation in v_mfma_scale_f32_*_f8f6f4.  Three kernels, for up to four rows a
// group (stream), some tens (block) and long groups (tile); which one is at the end of the file, with both sides'
// times.
#include <cmath>

#include "common.hpp"
#include "launch.hpp"
#include "ring.hpp"

namespace gg {
namespace fp4 {
using namespace ring;

// Lane layout of the 4-bit operands (checked on the GPU against a 64-bit product, all four scale bytes):
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds row (or column) l % 16, the 32 elements of k block l / 16
//   of the 128-wide slice, 16 bytes in the low half of the operand, and that block's scale in byte `op_sel`
//   of its scale register.  Result element e of lane l is C[4 (l / 16) + e][l % 16].
// v_mfma_scale_f32_32x32x64_f8f6f4: row l % 32, k block l / 32; result as the 32x32 bf16 instruction.
constexpr int kFp4 = 4;   // operand format selector of e2m1
__device__ inline i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// 16 (or 4) bytes a lane straight into LDS, as ring.hpp's loads, with the wait states that this target asks
// for: one between a scalar write of m0 and the load that takes its LDS address from it, five between a vector
// instruction's write of a scalar register (a readfirstlane, or a spilled descriptor's reload) and a load that
// reads it.  The compiler puts them in where it sees both instructions; it does not look into asm.
__device__ inline void load16(i32x4 r, uint32_t lds_addr, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds_addr), "v"(off), "s"(r) : "memory", "m0");
}
__device__ inline void load4(i32x4 r, uint32_t lds_addr, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds_addr), "v"(off), "s"(r) : "memory", "m0");
}

constexpr int kPanel = 256;           // elements along k of one scale panel
constexpr int kRowBytes = kPanel / 2; // code bytes of one row of a panel: one cache line

// The 16-byte chunks of a 128-byte LDS row are XORed by (row >> 1) & 7: 16 consecutive rows of one chunk
// then cover the 64 banks once.
__device__ inline int swizzle(int row) { return (row >> 1) & 7; }

// Row tile of a launch: which group, which rows.
struct RowTile {
    int grp;     // -1: nothing to do; -2: rows past the groups' total (zeros)
    int row0, rows;
};

// Row tile number `slot` among all groups' tiles of `tile_rows` rows, found by every wave for itself: lane i
// sums groups PER i .. PER i + PER - 1 (clamped as build_tables clamps them), a wave scan gives the tile
// offsets, and the lane that holds the slot walks its own groups.  Tiles past the last group's are the rows
// from the covered total to m.  Returns the GG_DEV_* bits in *flags.
template <int PER>
__device__ inline RowTile find_row_tile(const int32_t* __restrict__ sizes, int g, int m, int tile_rows, int slot, uint32_t* flags) {
    const int l = threadIdx.x & 63;
    int v[PER];
    long long sum = 0;
    bool neg = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int h = PER * l + i;
        const int x = h < g ? sizes[h] : 0;
        neg |= x < 0;
        v[i] = x < 0 ? 0 : x;
        sum += v[i];
    }
    const long long before = wave_inclusive_scan(sum) - sum;
    const long long total = __shfl(before + sum, 63, 64);
    const int covered = (int)(total < m ? total : m);
    int tiles = 0;
    long long p = before;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int st = (int)(p < m ? p : m), en = (int)(p + v[i] < m ? p + v[i] : m);
        tiles += (en - st + tile_rows - 1) / tile_rows;
        p += v[i];
    }
    int inc = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(inc, d, 64);
        if (l >= d) inc += u;
    }
    const int all = __shfl(inc, 63, 64);
    *flags = (__ballot(neg) ? GG_DEV_NEGATIVE_SIZE : 0u) | (total > m ? GG_DEV_SUM_EXCEEDS_M : 0u);
    RowTile r{-1, 0, 0};
    if (slot >= all) {
        const long long at = covered + (long long)(slot - all) * tile_rows;
        if (at < m) r = {-2, (int)at, (int)(m - at < tile_rows ? m - at : tile_rows)};
        return r;
    }
    int grp = 0, row0 = 0, rows = 0, first = inc - tiles;
    p = before;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int st = (int)(p < m ? p : m), en = (int)(p + v[i] < m ? p + v[i] : m);
        const int nt = (en - st + tile_rows - 1) / tile_rows;
        if (slot >= first && slot < first + nt) {
            grp = PER * l + i;
            row0 = st + (slot - first) * tile_rows;
            rows = min(tile_rows, en - row0);
        }
        first += nt;
        p += v[i];
    }
    const uint64_t owner = __ballot(rows > 0);   // exactly one lane
    const int src = __ffsll((unsigned long long)owner) - 1;
    r.grp = __builtin_amdgcn_readfirstlane(__shfl(grp, src, 64));
    r.row0 = __builtin_amdgcn_readfirstlane(__shfl(row0, src, 64));
    r.rows = __builtin_amdgcn_readfirstlane(__shfl(rows, src, 64));
    return r;
}

// row tiles (and tiles of rows past the total) that any group_sizes can give
inline int64_t slot_bound(const Fp4Params& p, int tile_rows) { return (p.g < p.m ? p.g : p.m) + (int64_t)p.m / tile_rows + 1; }

// scale bytes of k blocks at and past `valid` (of the four in the word) cleared
__device__ inline uint32_t keep_bytes(uint32_t w, int valid) { return valid >= 4 ? w : valid <= 0 ? 0u : w & ((1u << (8 * valid)) - 1u); }

__device__ inline void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, 0.f); }
__device__ inline void store1(float* p, float v) { *p = v; }

// Four consecutive columns of one row; `left` = columns of the row from here on.  A row begins where n puts it,
// so the stores are aligned to an element only (the target's global memory takes that).
typedef i32x2 __attribute__((aligned(2))) i32x2_any;
typedef i32x4 __attribute__((aligned(2))) i32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
template <typename OutT>
__device__ inline void store4(OutT* o, f32x4 v, int left) {
    if (left >= 4) {
        if constexpr (sizeof(OutT) == 2) *(i32x2_any*)o = i32x2{(int)pack_bf16(v[0], v[1]), (int)pack_bf16(v[2], v[3])};
        else *(f32x4_any*)o = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) store1(o + e, v[e]);
    }
}

// Stream kernel, for few rows a group: a workgroup holds the rows of one row tile (up to 16, all of k) in LDS
// and its four waves each stream weights past them, 16 columns (a column tile) at a time, through a private
// LDS ring of D panels (2 KiB of codes and their scales, loaded straight into LDS).  A wave's stream runs
// through its column tiles without a stop and without a barrier; results leave as each tile ends.  Bound by
// memory: what counts is the bytes in flight, 4 D panels of 2 KiB a workgroup and two workgroups a CU (D = 5
// measured the same as 4).  64 tokens at 4 of 128 experts, k = 2880, n = 5760: 177 us, 5.5 TB/s of codes and
// scales; one token at 2 of 8, k = 4096, n = 14336: 14.1 us, 4.4 TB/s with the launch and the first loads.
namespace stream {
constexpr int WAVES = 4;
constexpr int WPANEL = 16 * kRowBytes, SLOT = WPANEL + 256;   // scales: 128 bytes, loaded 4 bytes a lane
constexpr int LOADS = 3, D = 4;
constexpr int kMaxRowBytes = 28 * 1024;   // rows of one tile in LDS, so that a CU holds two workgroups

template <int PER, typename OutT>
__global__ __launch_bounds__(64 * WAVES) void kernel(Fp4Params p, int splits, int xrows) {
    // rows: panel by panel [xrows][128 bytes], then scales [panels][16][8]; 1 KiB of slack, as lanes of rows
    // that are not there (their results are not stored) read on
    __shared__ __attribute__((aligned(16))) uint8_t smem[WAVES * D * SLOT + kMaxRowBytes + 1024];
    const int t = threadIdx.x, l = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int slot = blockIdx.x / splits, split = blockIdx.x % splits;
    uint32_t flags;
    const RowTile rt = find_row_tile<PER>(p.group_sizes, p.g, p.m, 16, slot, &flags);
    if (blockIdx.x == 0 && t == 0) *p.status = flags;
    if (rt.grp == -1) return;
    OutT* out = (OutT*)p.out;
    const int nct = (p.n + 15) >> 4;
    const int ct0 = (int)((int64_t)split * nct / splits), ct1 = (int)((int64_t)(split + 1) * nct / splits);
    if (rt.grp == -2) {
        const int c0 = 16 * ct0, width = min(16 * ct1, p.n) - c0;
        for (int i = t; i < width * rt.rows; i += 64 * WAVES) store1(out + (size_t)(rt.row0 + i / width) * p.n + c0 + i % width, 0.f);
        return;
    }
    const int rows = rt.rows, panels = (p.k + kPanel - 1) / kPanel, rb = p.k >> 1;
    uint8_t* xl = smem + WAVES * D * SLOT;
    uint8_t* xs = xl + panels * xrows * kRowBytes;

    // the wave's stream of (column tile, panel)
    const int tiles = ct1 - ct0 > wave ? (ct1 - ct0 - wave + WAVES - 1) / WAVES : 0;
    const uint32_t ring0 = lds_u32(smem) + (uint32_t)(wave * D * SLOT);
    const uint8_t* mine = smem + wave * D * SLOT;
    const int lr = l >> 3;
    const uint32_t byte0 = 16u * (uint32_t)((l & 7) ^ swizzle(lr)), byte1 = 16u * (uint32_t)((l & 7) ^ swizzle(8 + lr));
    const uint8_t* const wbase = p.rhs + (size_t)rt.grp * p.n * rb;
    const uint8_t* const sbase = p.rhs_scale + (size_t)rt.grp * panels * p.n * 8;
    int lc = 0, lp = 0;   // tile and panel to load next
    auto load = [&](int s) {
        const int col = 16 * (ct0 + wave + WAVES * lc), cols = min(16, p.n - col);
        const bool live = lc < tiles;
        const i32x4 rw = make_rsrc_v(wbase + (size_t)(live ? col : 0) * rb, live ? (uint32_t)cols * (uint32_t)rb : 0u);
        const i32x4 rs = make_rsrc_v(sbase + ((size_t)lp * p.n + (live ? col : 0)) * 8, live ? (uint32_t)cols * 8u : 0u);
        const uint32_t at = ring0 + (uint32_t)(s * SLOT), pb = (uint32_t)lp * kRowBytes;
        const bool ok0 = pb + byte0 < (uint32_t)rb, ok1 = pb + byte1 < (uint32_t)rb;   // chunks past k
        load16(rw, at, ok0 ? (uint32_t)lr * (uint32_t)rb + pb + byte0 : kOOB);
        load16(rw, at + 1024u, ok1 ? (uint32_t)(8 + lr) * (uint32_t)rb + pb + byte1 : kOOB);
        load4(rs, at + WPANEL, 4u * (uint32_t)l);
        if (++lp == panels) { lp = 0; ++lc; }
    };
#pragma unroll
    for (int s = 0; s < D; ++s) load(s);

    // the rows, once
    {
        const i32x4 rx = make_rsrc_v(p.lhs + (size_t)rt.row0 * rb, (uint32_t)rows * (uint32_t)rb);
        const uint32_t x0 = lds_u32(xl);
        for (int i = wave; i < panels * (xrows >> 3); i += WAVES) {
            const int panel = xrows == 8 ? i : i >> 1, half = xrows == 8 ? 0 : i & 1;
            const uint32_t b = (uint32_t)panel * kRowBytes + (half ? byte1 : byte0);
            load16(rx, x0 + 1024u * (uint32_t)i, b < (uint32_t)rb ? (uint32_t)(8 * half + lr) * (uint32_t)rb + b : kOOB);
        }
        for (int i = t; i < panels * 16; i += 64 * WAVES) {
            const int r = i & 15;
            uint64_t v = 0;
            if (r < rows) v = *(const uint64_t*)(p.lhs_scale + ((size_t)(i >> 4) * p.m + rt.row0 + r) * 8);
            *(uint64_t*)(xs + 8 * i) = v;
        }
        wait_vm<0>();
        __syncthreads();
    }

    const int r = l & 15, q = l >> 4;
    const uint32_t c0 = (uint32_t)(((2 * q) ^ swizzle(r)) << 4), c1 = c0 ^ 16u;   // chunks 2 q and 2 q + 1 of row r
    int s = 0;
    for (int c = 0; c < tiles; ++c) {
        f32x4 acc0 = {0.f, 0.f, 0.f, 0.f}, acc1 = {0.f, 0.f, 0.f, 0.f};
        for (int panel = 0; panel < panels; ++panel) {
            wait_vm<LOADS * (D - 1)>();   // the oldest panel is in LDS
            const uint8_t* w = mine + s * SLOT + r * kRowBytes;
            const uint8_t* x = xl + panel * (xrows * kRowBytes) + r * kRowBytes;
            const i32x4 w0 = *(const i32x4*)(w + c0), w1 = *(const i32x4*)(w + c1);
            const i32x4 y0 = *(const i32x4*)(x + c0), y1 = *(const i32x4*)(x + c1);
            const int valid = (p.k >> 5) - panel * 8 - 2 * q;   // the lane's k blocks inside k
            const uint32_t sw = keep_bytes(*(const uint16_t*)(mine + s * SLOT + WPANEL + r * 8 + 2 * q), valid);
            const uint32_t sx = keep_bytes(*(const uint16_t*)(xs + (panel * 16 + r) * 8 + 2 * q), valid);
            __builtin_amdgcn_s_waitcnt(0xc07f);   // the slot has been read (lgkmcnt(0)): it can be filled again
            __builtin_amdgcn_sched_barrier(0);
            load(s);
            s = s + 1 == D ? 0 : s + 1;
            acc0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w0), widen(y0), acc0, kFp4, kFp4, 0, (int)sw, 0, (int)sx);
            acc1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w1), widen(y1), acc1, kFp4, kFp4, 1, (int)sw, 1, (int)sx);
        }
        const int col = 16 * (ct0 + wave + WAVES * c) + 4 * q;
        if (r < rows && col < p.n) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc0[e] + acc1[e];
            store4(out + (size_t)(rt.row0 + r) * p.n + col, v, p.n - col);
        }
    }
    wait_vm<0>();   // no load may still be writing LDS when the workgroup ends
}

inline int row_bytes(const Fp4Params& p) {
    const int panels = (p.k + kPanel - 1) / kPanel;
    return panels * ((p.m <= 8 ? 8 : 16) * kRowBytes + 128);
}

template <int PER>
hipError_t launch_per(const Fp4Params& p, int64_t grid, int splits, int xrows, hipStream_t s) {
    if (p.out_f32) hipLaunchKernelGGL((kernel<PER, float>), dim3((uint32_t)grid), dim3(64 * WAVES), 0, s, p, splits, xrows);
    else hipLaunchKernelGGL((kernel<PER, uint16_t>), dim3((uint32_t)grid), dim3(64 * WAVES), 0, s, p, splits, xrows);
    return hipGetLastError();
}
inline hipError_t launch(const Fp4Params& p, int cus, hipStream_t s) {
    const int nct = (p.n + 15) / 16;
    const int64_t slots = slot_bound(p, 16);
    // about eight workgroups a CU, none with fewer than a column tile a wave
    int64_t splits = (8 * (int64_t)cus + slots - 1) / slots;
    if (splits > nct / WAVES) splits = nct / WAVES;
    if (splits < 1) splits = 1;
    const int64_t grid = slots * splits;
    const int xrows = p.m <= 8 ? 8 : 16;
    if (p.g <= 64) return launch_per<1>(p, grid, (int)splits, xrows, s);
    if (p.g <= 256) return launch_per<4>(p, grid, (int)splits, xrows, s);
    return launch_per<16>(p, grid, (int)splits, xrows, s);
}
}  // namespace stream

// Block kernel, for some tens of rows a group and for every shape that the other two do not take: a workgroup
// walks a run of column tiles of one row tile, 64 rows x 128 columns each, as one stream of panels.  A panel
// (both operands' codes and scales) is loaded straight into one of D LDS slots, each wave an equal share; a
// panel that every wave has is read by all four, 64 rows x 32 columns of 32x32x64 instructions a wave, while
// the next D - 1 are on their way.  One barrier a panel, and two workgroups a CU cover each other's.  The
// weights are read once for 64 rows of their group, which leaves it bound by memory: a panel's instructions
// take 260 of the 2100 clocks in which a CU's share of the bandwidth brings its weights.  1500 rows of 32 groups,
// k = 2880, n = 1447, fp32: 22 us, 3.7 TB/s; 16 rows at each of 128 groups, k = 7168, n = 2048: 171 us, 5.9 TB/s.
// (Before it, 32 x 32 tiles with k split over the waves took 39 us for the first; tiles of 128 rows, for 64 to
// 200 rows a group, were 20 % to 50 % slower than the tile kernel or this one throughout.)
namespace block {
constexpr int ROWS = 64, COLS = 128, NT = 256, D = 3, SUB = 4, MI = ROWS / 32;
constexpr int W = COLS * kRowBytes, X = ROWS * kRowBytes, WS = COLS * 8, XS = ROWS * 8, SLOT = W + X + WS + XS;
constexpr int LOADS = 8;   // a wave's loads of a panel: 4 of weights, 2 of rows, 1 of each one's scales

template <int PER, typename OutT>
__global__ __launch_bounds__(NT, 2) void kernel(Fp4Params p, int splits, int run, int together) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[D * SLOT];
    const int t = threadIdx.x, l = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    int slot = blockIdx.x / splits, split = blockIdx.x % splits;
    if (together) {   // a group's row tiles at the same columns run side by side on one XCD and share the weights in its L2
        const int slots = gridDim.x / splits, v = xcd_virtual_id(blockIdx.x, gridDim.x);
        slot = v % slots;
        split = v / slots;
    }
    uint32_t flags;
    const RowTile rt = find_row_tile<PER>(p.group_sizes, p.g, p.m, ROWS, slot, &flags);
    if (blockIdx.x == 0 && t == 0) *p.status = flags;
    if (rt.grp == -1) return;
    OutT* out = (OutT*)p.out;
    const int nct = (p.n + COLS - 1) / COLS;
    const int ct0 = min(split * run, nct), ct1 = min(ct0 + run, nct);
    const int panels = (p.k + kPanel - 1) / kPanel, rb = p.k >> 1;
    if (rt.grp == -2 || panels == 0) {
        const int c0 = COLS * ct0, width = min(COLS * ct1, p.n) - c0;
        for (int i = t >> 6; i < rt.rows; i += NT / 64)
            for (int c = l; c < width; c += 64) store1(out + (size_t)(rt.row0 + i) * p.n + c0 + c, 0.f);
        return;
    }
    const int rows = rt.rows, tiles = ct1 - ct0;

    // the stream of (column tile, panel); a load brings eight rows, lane l row l / 8 into chunk place l % 8
    const uint32_t ring0 = lds_u32(smem);
    const int lr = l >> 3, lcol = 32 * wave + lr, lrow = 8 * MI * wave + lr;
    const uint32_t byte0 = 16u * (uint32_t)((l & 7) ^ (lr >> 1)), byte1 = byte0 ^ 64u;   // of even and odd eights
    const i32x4 rx = make_rsrc_v(p.lhs + (size_t)rt.row0 * rb, (uint32_t)rows * (uint32_t)rb);
    const uint8_t* const wbase = p.rhs + (size_t)rt.grp * p.n * rb;
    const uint8_t* const sbase = p.rhs_scale + (size_t)rt.grp * panels * p.n * 8;
    const uint8_t* const xbase = p.lhs_scale + (size_t)rt.row0 * 8;
    int lc = 0, lp = 0;   // tile and panel to load next
    auto load = [&](int s) {
        const bool live = lc < tiles;
        const int col = live ? COLS * (ct0 + lc) : 0, cols = live ? min(COLS, p.n - col) : 0;
        const i32x4 rw = make_rsrc_v(wbase + (size_t)col * rb, (uint32_t)cols * (uint32_t)rb);
        const i32x4 rws = make_rsrc_v(sbase + ((size_t)lp * p.n + col) * 8, (uint32_t)cols * 8u);
        const i32x4 rxs = make_rsrc_v(xbase + (size_t)lp * p.m * 8, live ? (uint32_t)rows * 8u : 0u);
        const uint32_t at = ring0 + (uint32_t)(s * SLOT), pb = (uint32_t)lp * kRowBytes;
        const bool ok0 = live && pb + byte0 < (uint32_t)rb, ok1 = live && pb + byte1 < (uint32_t)rb;   // chunks past k
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load16(rw, at + 1024u * (uint32_t)(4 * wave + i), (i & 1 ? ok1 : ok0) ? (uint32_t)(lcol + 8 * i) * (uint32_t)rb + pb + (i & 1 ? byte1 : byte0) : kOOB);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            load16(rx, at + W + 1024u * (uint32_t)(MI * wave + i), (i & 1 ? ok1 : ok0) ? (uint32_t)(lrow + 8 * i) * (uint32_t)rb + pb + (i & 1 ? byte1 : byte0) : kOOB);
        load4(rws, at + W + X + 256u * (uint32_t)wave, 256u * (uint32_t)wave + 4u * (uint32_t)l);
        load4(rxs, at + W + X + WS + 256u * (uint32_t)(wave & 1), 256u * (uint32_t)(wave & 1) + 4u * (uint32_t)l);   // (two waves bring the same)
        if (++lp == panels) { lp = 0; ++lc; }
    };
#pragma unroll
    for (int s = 0; s < D - 1; ++s) load(s);

    // fragments: lane l holds row l % 32 of a block of 32 and k blocks 4 (l / 32) + sub of the panel
    const int h = l >> 5, r = l & 31;
    const uint32_t chunk0 = (uint32_t)((4 * h) ^ ((l >> 1) & 7)) << 4;
    const uint32_t aw = (uint32_t)(32 * wave + r) * kRowBytes + chunk0, ax = W + (uint32_t)r * kRowBytes + chunk0;
    const uint32_t aws = W + X + (uint32_t)(32 * wave + r) * 8u + 4u * (uint32_t)h, axs = W + X + WS + (uint32_t)r * 8u + 4u * (uint32_t)h;
    const int blocks = (rows + 31) >> 5;
    int s = 0, ls = D - 1;
    for (int c = 0; c < tiles; ++c) {
        f32x16 acc[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;
        for (int panel = 0; panel < panels; ++panel) {
            // every wave's share of the oldest panel is in LDS, and the panel before it has been read
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS * (D - 2)) : "memory");
            load(ls);
            ls = ls + 1 == D ? 0 : ls + 1;
            const uint8_t* const at = smem + s * SLOT;
            s = s + 1 == D ? 0 : s + 1;
            i32x4 fw[SUB], fx[MI][SUB];
            const int valid = (p.k >> 5) - panel * 8 - 4 * h;   // the lane's four k blocks inside k
            const int sw = (int)keep_bytes(*(const uint32_t*)(at + aws), valid);
            int sx[MI];
#pragma unroll
            for (int e = 0; e < SUB; ++e) fw[e] = *(const i32x4*)(at + (aw ^ (uint32_t)(e << 4)));
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                sx[i] = (int)keep_bytes(*(const uint32_t*)(at + axs + 256 * i), valid);
#pragma unroll
                for (int e = 0; e < SUB; ++e) fx[i][e] = *(const i32x4*)(at + (ax ^ (uint32_t)(e << 4)) + 32 * i * kRowBytes);
            }
            // (the weights first, so that a lane holds four columns of one row)
            static_for<0, MI>([&](auto i_c) {
                constexpr int i = decltype(i_c)::value;
                if (i > 0 && i >= blocks) return;
                static_for<0, SUB>([&](auto e_c) {
                    constexpr int e = decltype(e_c)::value;
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(fw[e]), widen(fx[i][e]), acc[i], kFp4, kFp4, e, sw, e, sx[i]);
                });
            });
        }
        // element 4 q + u of block i: row 32 i + l % 32, column 8 q + 4 h + u of the wave's
        const int col = COLS * (ct0 + c) + 32 * wave + 4 * h;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int row = 32 * i + r;
            OutT* const o = out + (size_t)(rt.row0 + row) * p.n + col;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (row < rows && col + 8 * q < p.n) store4(o + 8 * q, f32x4{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]}, p.n - col - 8 * q);
        }
    }
    wait_vm<0>();   // no load may still be writing LDS when the workgroup ends
}

template <int PER>
hipError_t launch_per(const Fp4Params& p, int64_t grid, int splits, int run, int together, hipStream_t s) {
    if (p.out_f32) hipLaunchKernelGGL((kernel<PER, float>), dim3((uint32_t)grid), dim3(NT), 0, s, p, splits, run, together);
    else hipLaunchKernelGGL((kernel<PER, uint16_t>), dim3((uint32_t)grid), dim3(NT), 0, s, p, splits, run, together);
    return hipGetLastError();
}

inline hipError_t launch(const Fp4Params& p, int cus, hipStream_t s) {
    const int nct = (p.n + COLS - 1) / COLS;
    const int64_t slots = slot_bound(p, ROWS);
    // about eight workgroups a CU, or one for every column tile of every row tile
    int64_t run = slots * nct / (8 * (int64_t)cus);
    run = run > nct ? nct : run;
    run = run < 1 ? 1 : run;
    int64_t splits = (nct + run - 1) / run;
    splits = splits < 1 ? 1 : splits;   // (n = 0: the status word alone)
    const int together = p.m / p.g > ROWS && splits >= 8;   // (else an XCD's share could be mostly empty row tiles)
    const int64_t grid = together ? (slots * splits + 7) / 8 * 8 : slots * splits;   // (past the last split: nothing)
    if (p.g <= 64) return launch_per<1>(p, grid, (int)splits, (int)run, together, s);
    if (p.g <= 256) return launch_per<4>(p, grid, (int)splits, (int)run, together, s);
    return launch_per<16>(p, grid, (int)splits, (int)run, together, s);
}
}  // namespace block

// Tile kernel: 256 x 256 tiles, four waves of 128 x 128 (4 x 4 blocks of 32x32x64 instructions, the results
// in 256 accumulator registers), one workgroup a CU, each walking its tiles as one stream of panels (256
// along k).  A panel is 128 bytes of each of the tile's 512 rows, one cache line a row, and 4 KiB of scales,
// in one of two LDS slots.  While the instructions of panel c run, from registers, the operands of panel
// c + 1 come out of their slot into the registers that panel c has done with, and panel c + 2 is loaded into
// panel c's slot, which was emptied before panel c began: a load has all but the first MFMAs of a panel to
// arrive.  The stream runs on into the workgroup's next tile, so a tile begins with its first panel in
// registers and its second in LDS.  Between two tiles no matrix instruction runs: the results turn in LDS and go
// out as stores, of which only the last are still under way while the next tile's first panel is computed.
// 8192 rows of 8 groups, k = 4096, n = 14336: 266 us, 3600 TFLOP/s.  32768 rows of 256 very unequal groups,
// k = 7168, n = 2048: 505 us among other calls; in a row of twelve 498 to 592, median 564, as the chip lowers its
// clock: 4.5 and 4.0 TB/s, bound by memory.  8192 rows of 8 groups, n = 8192, which are four tiles a workgroup,
// with 3 / 8 / 16 / 64 panels: 57 / 81 / 147 / 500 us (4400 TFLOP/s): 1.8 to 2.1 us a panel, and 7 to 9 us a tile
// beside them, the launch among it.  Without its loads a panel takes 1.5: these instructions alone run at 6300
// TFLOP/s on random data and 8700 on zeros, with the operands' reads from LDS at 5700 to 6200 and 8800.  Loads
// spread over the first 31, 45, 52 or 60 of a panel's 64 instructions measured within 2 %, all before the first
// 2.0 us.
namespace tile {
constexpr int BM = 256, BN = 256, NT = 256, MI = 4, NJ = 4, SUB = 4;   // SUB: instructions along k of a panel
constexpr int OPER = 256 * kRowBytes;     // one operand's slot
constexpr int SC = 256 * 8;               // one operand's scales of a panel
// panels between the starts of neighbouring column tiles.  2 / 0, in us, at 8192 rows of 8 groups, n = 8192: k = 768
// 57.4 / 56.3, 1024 60.0 / 61.2, 2048 80.9 / 82.4, 2880 113.1 / 114.6, 4096 147.0 / 148.0, 7168 237.1 / 234.3, 8192
// 266.9 / 264.7, 16384 499.5 / 500.8; (32, 2880, 5760) x 512 187.2 / 190.6; (256, 7168, 2048) x 128 439.9 / 443.0:
// at most 2 % either way, and more of the shapes above faster with 2
constexpr int ROT = 2;
constexpr int LOADS = 17;                 // a wave's loads of a panel: 1 KiB of scales, 8 + 8 of eight rows
constexpr int READ = 15;                  // MFMA of a panel after which the next panel's reads begin
constexpr int load_step(int d) { return d * 31 / LOADS; }   // MFMA after which load d goes out
constexpr int loads_before(int step) {
    int n = 0;
    while (n < LOADS && load_step(n) <= step) ++n;
    return n;
}
struct alignas(16) Smem {
    uint8_t a[2][OPER];
    uint8_t b[2][OPER];
    uint8_t sc[2][2 * SC];                // row scales, column scales
    Tables tab;
};

// A wave-uniform value in a scalar register.  (Where the compiler knows a value to be uniform it folds
// readfirstlane away; a value read from LDS, or one carried around a loop, then stays in vector registers, and
// with it the descriptors that the loads below need in scalar ones.  So the value is made opaque first.)
__device__ inline int scalar(int v) {
    asm volatile("" : "+v"(v));
    return __builtin_amdgcn_readfirstlane(v);
}

// the largest h with tile_off[h] <= t (find_group, in two steps of one read a lane)
__device__ inline int find_group_wave(const int* tile_off, int g, int t) {
    const int l = threadIdx.x & 63;
    const int c = tile_off[min(16 * l, g)];
    const int blk = __popcll(__ballot(16 * l < g && c <= t)) - 1;
    const int h = 16 * blk + (l & 15);
    const int f = tile_off[min(h, g)];
    return __builtin_amdgcn_readfirstlane(16 * blk + __popcll(__ballot(l < 16 && h < g && f <= t)) - 1);
}

// WHOLE: rows of the output are multiples of 16 bytes and aligned so
template <typename OutT, bool WHOLE>
__global__ __launch_bounds__(NT, 1) void kernel(Fp4Params p) {
    __shared__ Smem sm;
    const int t = threadIdx.x, l = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r0w = 128 * (wave >> 1), c0w = 128 * (wave & 1);
    const int ntn = cdiv(p.n, BN);
    int gemm_tiles, covered;
    build_tables<NT>(p.group_sizes, p.g, p.m, BM, ntn, sm.tab, &gemm_tiles, &covered);
    gemm_tiles = scalar(gemm_tiles);
    covered = scalar(covered);
    if (blockIdx.x == 0 && t == 0) *p.status = sm.tab.flags;
    const int rb = p.k >> 1, panels = (p.k + kPanel - 1) / kPanel;
    OutT* const out = (OutT*)p.out;
    constexpr int OSZ = sizeof(OutT), PIECE = 16 / OSZ, JS = OSZ == 2 ? NJ : NJ / 2;   // JS: blocks of a 256-byte strip
    const int first = xcd_virtual_id(blockIdx.x, gridDim.x);

    struct Info { int row0, rows, col0, turn0; };   // turn0: the panel that the tile begins with
    // the load stream's tile: rows, weights, and the scales this wave loads, as the parts of descriptors (whole
    // ones, carried around the loop, end up in vector registers)
    struct Desc {
        int lo, hi, bytes;
        __device__ void set(const void* base, uint32_t n) {
            lo = (int)(uint32_t)(uintptr_t)base;
            hi = (int)((uint32_t)((uintptr_t)base >> 32) & 0xffffu);
            bytes = (int)n;
        }
        __device__ i32x4 get() const { return i32x4{lo, hi, bytes, kRsrcWord3}; }
        __device__ void pin() { lo = scalar(lo); hi = scalar(hi); bytes = scalar(bytes); }   // into scalar registers
    };
    Desc ra, rw, rs;
    auto decode = [&](int tile) {
        const int grp = find_group_wave(sm.tab.tile_off, p.g, tile);
        const int local = tile - scalar(sm.tab.tile_off[grp]);
        int row0 = scalar(sm.tab.row_off[grp]);
        const int size = scalar(sm.tab.row_off[grp + 1]) - row0;
        const int mtg = cdiv(size, BM);
        int mt, nt;
        if (size <= p.n) { mt = local % mtg; nt = local / mtg; }   // neighbours share the larger operand
        else { nt = local % ntn; mt = local / ntn; }
        // Rows are a multiple of a large power of two apart, so that one panel of a tile lies in few of L2's
        // channels: tiles side by side begin at different panels and go around, those with the same weights at
        // the same one.
        Info i{row0 + mt * BM, min(BM, size - mt * BM), nt * BN, (ROT * nt) % panels};
        ra.set(p.lhs + (size_t)i.row0 * rb, (uint32_t)i.rows * (uint32_t)rb);
        rw.set(p.rhs + ((size_t)grp * p.n + i.col0) * rb, (uint32_t)min(BN, p.n - i.col0) * (uint32_t)rb);
        // a panel's scales of rows past the tile belong to rows that are not stored
        const uint8_t* s = wave < 2 ? p.lhs_scale + (size_t)i.row0 * 8 : p.rhs_scale + ((size_t)grp * panels * p.n + i.col0) * 8;
        const int rows = wave < 2 ? p.m : p.n, at = wave < 2 ? i.row0 : i.col0;
        rs.set(s, ((uint32_t)panels * (uint32_t)rows - (uint32_t)at) * 8u);
        return i;
    };

    // Load number d of the stream's panel lp: the scales, then (counting on from 0) d < 8 rows 64 wave + 8 d .. + 7,
    // d < 16 the same of the weights.  The scales come first, before a panel's instructions: their load is behind a
    // branch, and the compiler moves what instructions it can past a branch, away from the loads that they were
    // to be spread among.  Lane l brings row l / 8 of the eight, chunk (l % 8) ^ swizzle(row); the swizzle of row
    // 64 wave + 8 d + l / 8 is (4 d + l / 16) % 8.  v: lane offsets for even and odd d; in a last panel that k
    // does not fill, the chunks past k are out of range and read as zeros.
    const int lc = (l & 7) ^ (l >> 4);
    const uint32_t v0 = (uint32_t)(l >> 3) * (uint32_t)rb + 16u * (uint32_t)lc, v1 = (uint32_t)(l >> 3) * (uint32_t)rb + 16u * (uint32_t)(lc ^ 4);
    const int in_last = rb - (panels - 1) * kRowBytes;   // code bytes of the last panel
    const uint32_t vt0 = 16 * lc < in_last ? v0 : kOOB, vt1 = 16 * (lc ^ 4) < in_last ? v1 : kOOB;
    const uint32_t lds_a = lds_u32(&sm.a[0][0]), lds_b = lds_u32(&sm.b[0][0]), lds_s = lds_u32(&sm.sc[0][0]);
    const uint32_t srows = (uint32_t)(wave < 2 ? p.m : p.n) * 8u;
    uint32_t lslot = 0, past = 0;   // past: set once the stream has no more tiles, its loads then read nothing
    auto issue = [&](auto d_c, int lp) {
        constexpr int d = decltype(d_c)::value - 1;
        if constexpr (d >= 0) {
            const bool last = lp == panels - 1;
            const uint32_t v = d & 1 ? (last ? vt1 : v1) : (last ? vt0 : v0);
            const uint32_t s = (uint32_t)(64 * wave + 8 * (d & 7)) * (uint32_t)rb + (uint32_t)lp * kRowBytes + past;
            load16(d < 8 ? ra.get() : rw.get(), (d < 8 ? lds_a : lds_b) + lslot * OPER + (uint32_t)(8 * wave + (d & 7)) * 1024u, v + s);
        } else {
            const uint32_t to = lds_s + lslot * (2 * SC) + (uint32_t)wave * 1024u, from = (uint32_t)lp * srows + past + (uint32_t)(wave & 1) * 1024u;
            if (lp == panels - 1 && ((rs.bytes - lp * (int)srows) & 8)) {
                // the array may end 8 bytes into a 16-byte piece: 4 bytes a lane (the waits count the fewer loads)
#pragma unroll
                for (uint32_t e = 0; e < 1024; e += 256) load4(rs.get(), to + e, from + e + 4u * (uint32_t)l);
            } else {
                load16(rs.get(), to, from + 16u * (uint32_t)l);
            }
        }
    };

    // Fragments: lane l holds row l % 32 of a block and k blocks 4 (l / 32) + sub of the panel, one chunk and
    // one scale byte each; the four scale bytes are one word.  The chunk's place is (4 (l / 32) + sub) ^
    // swizzle(l), so a sub-slice's and a slot's address differ from the lane's own in single bits, and the
    // blocks of 32 rows by constants.
    const int h = l >> 5;
    const uint32_t chunk0 = (uint32_t)((4 * h) ^ ((l >> 1) & 7)) << 4;
    const uint32_t la = (uint32_t)(r0w + (l & 31)) * kRowBytes + chunk0, lb = (uint32_t)(c0w + (l & 31)) * kRowBytes + chunk0;
    const uint32_t lsa = lds_s + (uint32_t)(r0w + (l & 31)) * 8u + 4u * (uint32_t)h, lsb = lds_s + SC + (uint32_t)(c0w + (l & 31)) * 8u + 4u * (uint32_t)h;
    i32x4 fa[SUB][MI], fb[SUB][NJ], ta[MI], tb[NJ];   // ta, tb: the next panel's last sub-slice, which is read ahead of its turn
    int sa[MI], sb[NJ], na[MI], nb_[NJ];
    uint32_t rslot = 0, aa = 0, ab = 0;   // the slot that is read, and the addresses of the sub-slice that is
    auto aim = [&](int s) {
        const uint32_t k = rslot * OPER ^ (uint32_t)(s << 4);
        aa = lds_a + (la ^ k);
        ab = lds_b + (lb ^ k);
        asm volatile("" : "+v"(aa), "+v"(ab));   // kept as one address each, or every block's is computed and held
    };
    auto read_a = [&](i32x4& f, int i) { f = *(const __attribute__((address_space(3))) i32x4*)(uintptr_t)(aa + (uint32_t)(32 * i * kRowBytes)); };
    auto read_b = [&](i32x4& f, int j) { f = *(const __attribute__((address_space(3))) i32x4*)(uintptr_t)(ab + (uint32_t)(32 * j * kRowBytes)); };
    const int tail_valid = (p.k >> 5) - 8 * (panels - 1) - 4 * h;
    auto aim_scales = [&] {
        aa = lsa + rslot * (2 * SC);
        ab = lsb + rslot * (2 * SC);
        asm volatile("" : "+v"(aa), "+v"(ab));
    };
    auto read_sa = [&](int i) { na[i] = *(const __attribute__((address_space(3))) int*)(uintptr_t)(aa + (uint32_t)(32 * i * 8)); };
    auto read_sb = [&](int j) { nb_[j] = *(const __attribute__((address_space(3))) int*)(uintptr_t)(ab + (uint32_t)(32 * j * 8)); };
    auto take_scales = [&](int panel) {   // of the panel whose fragments were read last
        const uint32_t keep = panel == panels - 1 ? keep_bytes(~0u, tail_valid) : ~0u;
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[i] = na[i] & (int)keep;
#pragma unroll
        for (int j = 0; j < NJ; ++j) sb[j] = nb_[j] & (int)keep;
    };
    // for every wave: the panel after the one that is computed has arrived (its loads are older than the YOUNGER
    // youngest), and: its slot has been read
    auto arrived = [&](auto younger_c) {
        constexpr int YOUNGER = decltype(younger_c)::value;
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(YOUNGER < 63 ? YOUNGER : 63) : "memory");
    };
    auto emptied = [&] { lds_barrier(); };

    if (first < gemm_tiles) {
        Info cur = decode(first);
        auto issue_some = [&](auto b_c, auto e_c, int lp) {
            asm volatile("" : "+s"(lp));   // (or the offsets of a fixed panel are all computed ahead and held)
            static_for<decltype(b_c)::value, decltype(e_c)::value>([&](auto d_c) { issue(d_c, lp); });
        };
        auto issue_all = [&](int lp) {
            issue_some(std::integral_constant<int, 0>{}, std::integral_constant<int, LOADS>{}, lp);
            lslot ^= 1;
        };
        auto around = [&](int panel) { return panel < panels ? panel : panel - panels; };
        issue_all(around(cur.turn0));
        issue_all(around(cur.turn0 + 1));
        wait_vm<LOADS>();
        lds_barrier();
        static_for<0, SUB>([&](auto s_c) {
            aim(s_c);
            static_for<0, MI>([&](auto i_c) { read_a(s_c == SUB - 1 ? ta[i_c] : fa[s_c][i_c], i_c); });
            static_for<0, NJ>([&](auto j_c) { read_b(s_c == SUB - 1 ? tb[j_c] : fb[s_c][j_c], j_c); });
        });
        aim_scales();
        static_for<0, MI>([&](auto i_c) { read_sa(i_c); });
        static_for<0, NJ>([&](auto j_c) { read_sb(j_c); });
        emptied();
        take_scales(cur.turn0);
        rslot = 1;
        issue_all(around(cur.turn0 + 2));
        bool stored = false;   // the tile before left all of its STORES
        for (int tile = first; tile < gemm_tiles;) {
        Info next = cur;
        const int blocks = max(0, min(MI, cdiv(cur.rows - r0w, 32)));
        tile += gridDim.x;
        with_nb<2>((blocks + 1) >> 1, [&](auto nb_c) {
            constexpr int NB = 2 * decltype(nb_c)::value;
            f32x16 acc[NB > 0 ? NB : 1][NJ];
            constexpr int STORES = MI * (NJ / JS) * 8;   // a wave's of a whole tile
            // One panel: 16 steps a sub-slice, each at most one MFMA and the reads and loads that go with it.
            // FIRST: the tile's first panel, whose turn and loads are done already.  follow: the panel after it,
            // lp: the panel to load.
            auto panel = [&](auto first_c, int follow, int lp) {
                constexpr bool FIRST = decltype(first_c)::value;
                if constexpr (!FIRST) issue(std::integral_constant<int, 0>{}, lp);
                __builtin_amdgcn_sched_barrier(0);
                static_for<0, SUB>([&](auto s_c) {
                    constexpr int S = decltype(s_c)::value;
                    static_for<0, 16>([&](auto m_c) {
                        constexpr int M = decltype(m_c)::value;
                        constexpr int I = M >> 2, J = M & 3;
                        if constexpr (I < NB) {
                            const f32x16 zero = {};
                            // (the weights first, so that a lane holds columns of one row)
                            acc[I][J] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(fb[S][J]), widen(fa[S][I]), FIRST && S == 0 ? zero : acc[I][J], kFp4,
                                                                                        kFp4, S, sb[J], S, sa[I]);
                        }
                        // the last sub-slice, read during the panel before, to its place
                        if constexpr (S == 0 && M < 4) { fa[SUB - 1][M] = ta[M]; fb[SUB - 1][M] = tb[M]; }
                        constexpr int G = 16 * S + M;
                        // the loads, spread over the first half (a load takes a compute unit's address path 16
                        // clocks, so the four waves' go out no faster than one each in 64)
                        if constexpr (!FIRST) static_for<1, LOADS>([&](auto d_c) { if constexpr (load_step(decltype(d_c)::value) == G) issue(d_c, lp); });
                        // the next panel's reads, spread over the rest: its loads have had a panel and a quarter to
                        // arrive, and are older than those just begun
                        if constexpr (G == READ) {
                            if constexpr (!FIRST) {
                                arrived(std::integral_constant<int, loads_before(READ)>{});
                            } else if (stored) {
                                arrived(std::integral_constant<int, LOADS + STORES>{});
                            } else {
                                arrived(std::integral_constant<int, LOADS>{});
                            }
                        }
                        if constexpr (G >= 16 && G < 32) {
                            constexpr int K = G & 15;
                            if constexpr ((K & 7) == 0) aim(0);
                            if constexpr ((K & 7) == 4) aim(SUB - 1);
                            if constexpr (K < 4) read_a(fa[0][K], K);
                            else if constexpr (K < 8) read_a(ta[K & 3], K & 3);
                            else if constexpr (K < 12) read_b(fb[0][K & 3], K & 3);
                            else read_b(tb[K & 3], K & 3);
                        }
                        if constexpr (G >= 32 && G < 48) {
                            constexpr int K = G & 15;
                            if constexpr (K == 0) aim(1);
                            if constexpr (K == 8) aim_scales();
                            if constexpr (K < 4) read_a(fa[1][K], K);
                            else if constexpr (K < 8) read_b(fb[1][K & 3], K & 3);
                            else if constexpr (K < 12) read_sa(K & 3);
                            else read_sb(K & 3);
                        }
                        if constexpr (G >= 48 && G < 56) {
                            if constexpr (G == 48) aim(2);
                            if constexpr (G < 52) read_a(fa[2][G & 3], G & 3);
                            else read_b(fb[2][G & 3], G & 3);
                        }
                        if constexpr (G == 60) emptied();
                        __builtin_amdgcn_sched_barrier(0);
                    });
                });
                take_scales(follow);
                rslot ^= 1;
                if constexpr (!FIRST) lslot ^= 1;
            };
            int follow = around(cur.turn0 + 1), lp = around(cur.turn0 + 2);
            panel(std::true_type{}, follow, 0);
            // the tile's panels but the first and the last two load the panel two after, the last two the next
            // tile's first two
            int left = panels - 3;
            for (int half = 0; half < 2; ++half) {
                ra.pin(); rw.pin(); rs.pin();
                for (; left > 0; --left) {
                    follow = half && left == 1 ? next.turn0 : around(follow + 1);
                    lp = around(lp + 1);
                    panel(std::false_type{}, follow, lp);
                }
                if (half == 0) {
                    if (tile < gemm_tiles) next = decode(tile);
                    else past = kOOB;
                    lp = next.turn0 - 1;
                    left = 2;
                }
            }
        ra.pin(); rw.pin(); rs.pin();
        // The slot that has just been emptied takes the panel after the next: its rows and scales at once, its
        // weights once the results have passed through their place (8 KiB a wave, the part that its own loads fill).
        const int lp2 = around(next.turn0 + 2);
        issue_some(std::integral_constant<int, 0>{}, std::integral_constant<int, 9>{}, lp2);
        // Results: element 4 q + u of block (i, j) is row 32 i + l % 32, column 32 j + 8 q + 4 h + u.  They turn in
        // LDS, 256 bytes of 32 rows at a time (16-byte pieces XORed by the row), and leave as whole lines.
        uint8_t* const strip = &sm.b[0][0] + lslot * OPER + (uint32_t)wave * 8192u;
        const rsrc_t ro = make_rsrc(out + (size_t)cur.row0 * p.n, (uint32_t)cur.rows * (uint32_t)p.n * (uint32_t)OSZ);
        const uint32_t row_bytes = (uint32_t)p.n * (uint32_t)OSZ;
        // (lane parts of the addresses, opaque: every piece's would else be computed ahead and held)
        uint32_t put = lds_u32(strip) + (uint32_t)(l & 31) * 256u, turned = (uint32_t)(l & 15) << 4, take = lds_u32(strip) + (uint32_t)(l >> 4) * 256u, srow = (uint32_t)(l >> 4) << 4;
        asm volatile("" : "+v"(put), "+v"(turned), "+v"(take), "+v"(srow));
        static_for<0, NB * (NJ / JS)>([&](auto is_c) {
            constexpr int i = decltype(is_c)::value / (NJ / JS), j0 = decltype(is_c)::value % (NJ / JS) * JS;
            if (NB < MI && i >= blocks) return;   // (whole tiles' stores are counted: see arrived)
            static_for<0, JS>([&](auto j_c) {
                static_for<0, 4>([&](auto q_c) {
                    constexpr int j = decltype(j_c)::value, q = decltype(q_c)::value;
                    const f32x16& c = acc[i][j0 + j];
                    if constexpr (OSZ == 2) {
                        const i32x2 v = {(int)pack_bf16(c[4 * q], c[4 * q + 1]), (int)pack_bf16(c[4 * q + 2], c[4 * q + 3])};
                        *(__attribute__((address_space(3))) i32x2*)(uintptr_t)(put + (((4 * j + q) << 4) ^ turned) + 8 * h) = v;
                    } else {
                        *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(put + (((uint32_t)(8 * j + 2 * q + h) << 4) ^ turned)) = f32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
                    }
                });
            });
            const int col = cur.col0 + c0w + 32 * j0 + PIECE * (l & 15);
            uint32_t off = (uint32_t)(r0w + 32 * i + (int)(srow >> 4)) * row_bytes + (uint32_t)col * (uint32_t)OSZ;
#pragma unroll
            for (int r = 0; r < 32; r += 4) {
                // row r + l / 16, whose pieces are XORed by its low four bits
                const i32x4 v = *(const __attribute__((address_space(3))) i32x4*)(uintptr_t)(take + 256u * r + (turned ^ (srow + ((r & 15) << 4))));
                if constexpr (WHOLE) {
                    bstore(ro, col < p.n ? off : kOOB, v);
                } else if (r0w + 32 * i + r + (int)(srow >> 4) < cur.rows) {
                    uint8_t* const o = (uint8_t*)out + (size_t)cur.row0 * row_bytes + off;
                    if (col + PIECE <= p.n) {
                        *(i32x4_any*)o = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) {
                            if (col + e >= p.n) break;
                            if constexpr (OSZ == 2) *(uint16_t*)(o + 2 * e) = (uint16_t)((uint32_t)v[e >> 1] >> (16 * (e & 1)));
                            else *(int*)(o + 4 * e) = v[e & 3];
                        }
                    }
                }
                off += 4 * row_bytes;
            }
        });
        __builtin_amdgcn_s_waitcnt(0xc07f);   // the strip has been read (lgkmcnt(0))
        __builtin_amdgcn_sched_barrier(0);
        issue_some(std::integral_constant<int, 9>{}, std::integral_constant<int, LOADS>{}, lp2);
        lslot ^= 1;
        stored = WHOLE && NB == MI;
        });
        cur.row0 = scalar(next.row0); cur.rows = scalar(next.rows); cur.col0 = scalar(next.col0); cur.turn0 = scalar(next.turn0);
    }
    wait_vm<0>();   // no load may still be writing LDS when the workgroup ends
    }
    // rows past the groups' total
    const size_t lo = (size_t)covered * p.n, hi = (size_t)p.m * p.n;
    for (size_t i = lo + (size_t)blockIdx.x * NT + t; i < hi; i += (size_t)gridDim.x * NT) store1(out + i, 0.f);
}
}  // namespace tile

// 32-bit offsets of the tile kernel's descriptors, and at least three panels, as two are loaded ahead.  (Long groups
// of one or two panels go to the block kernel, whose stores of 8 or 16 bytes a lane bound it there: 8192 rows of 8
// groups, n = 7168, take 59 us at k = 256 and 72 at k = 512, 2.2 and 2.5 times what their bytes ask for.)
inline bool tile_ok(const Fp4Params& p) {
    const int64_t panels = (p.k + kPanel - 1) / kPanel;
    const int64_t tiles = ((int64_t)p.m / tile::BM + p.g + 1) * ((p.n + tile::BN - 1) / tile::BN);
    return p.k > 2 * kPanel && (int64_t)256 * (p.k >> 1) < (int64_t(1) << 30) && (int64_t)256 * p.n * 4 < (int64_t(1) << 31) &&
           panels * p.m * 8 < (int64_t(1) << 31) && panels * p.n * 8 < (int64_t(1) << 31) && tiles < (int64_t(1) << 30);
}

inline hipError_t launch_tile(const Fp4Params& p, int cus, hipStream_t s) {
    const int64_t tiles = ((int64_t)p.m / tile::BM + (p.g < p.m ? p.g : p.m)) * ((p.n + tile::BN - 1) / tile::BN);
    const int grid = (int)(tiles < cus ? (tiles < 1 ? 1 : tiles) : cus);
    const bool whole = ((uintptr_t)p.out & 15) == 0 && (p.n * (p.out_f32 ? 4 : 2)) % 16 == 0;
    if (p.out_f32) {
        if (whole) hipLaunchKernelGGL((tile::kernel<float, true>), dim3(grid), dim3(tile::NT), 0, s, p);
        else hipLaunchKernelGGL((tile::kernel<float, false>), dim3(grid), dim3(tile::NT), 0, s, p);
    } else {
        if (whole) hipLaunchKernelGGL((tile::kernel<uint16_t, true>), dim3(grid), dim3(tile::NT), 0, s, p);
        else hipLaunchKernelGGL((tile::kernel<uint16_t, false>), dim3(grid), dim3(tile::NT), 0, s, p);
    }
    return hipGetLastError();
}

// Tile or block kernel, by the times that their tiles' numbers and panels give (a host knows the groups' mean
// size only, rows past the last group among it: a group of mean size has a half-filled tile more than it fills, and
// at least one).  In us on 256
// CUs: the tile kernel's CUs take ceil(tiles / CUs) tiles each, 6 and 1.4 to 2.1 a panel with the tile's rows,
// the block kernel's 1.6 and 0.7 a panel for each of its tiles / CUs.  Measured, block / tile, at (groups, k, n) x
// rows a group: (32, 2880, 2880) x 48 45 / 54, x 64 51 / 58, x 112 66 / 61; (8, 4096, 14336) x 48 53 / 63,
// x 112 86 / 68; (128, 7168, 2048) x 32 179 / 184, x 48 204 / 192, x 80 310 / 203; few long groups, which are few
// tiles, (1, 6688, 2752) x 783 32 / 56, (8, 6400, 1344) x 272 26 / 47; (16, 1184, 1600) x 927 60 / 35.
// Where the mean says little the choice can miss: 512 rows that are all at one of 256 groups, k = 2880, n = 5760,
// take the stream kernel, 46 us against a floor of 3; 2048 rows at 8 of 64 groups of k = n = 4096 the block kernel,
// 43 us against 20.
inline bool tile_faster(const Fp4Params& p, int cus) {
    const double used = p.g < p.m ? p.g : p.m, per = p.m / used, panels = (p.k + kPanel - 1) / kPanel;
    const double t = used * fmax(1., per / tile::BM + .5) * ((p.n + tile::BN - 1) / tile::BN);
    const double b = used * fmax(1., per / block::ROWS + .5) * ((p.n + block::COLS - 1) / block::COLS);
    return ceil(t / cus) * (6. + (1.4 + .7 * fmin(1., per / tile::BM)) * panels) < b / cus * (1.6 + .7 * panels);
}

}  // namespace fp4

bool ragged_m_fp4_grid_ok(const Fp4Params& p) {
    // Column indices past n must not leave 32 bits either.  The block kernel's workgroups are at most its row tiles
    // and 16 more a compute unit (up to 1024 of them); that many keep m below 2^30, so that rounding a group's rows
    // up to whole tiles stays in 32 bits too.
    return p.n <= INT32_MAX - 256 && fp4::slot_bound(p, 16) * ((p.n + 15) / 16) <= INT32_MAX && (int64_t)128 * (p.k >> 1) < (int64_t(1) << 31) &&
           fp4::slot_bound(p, fp4::block::ROWS) + 16 * 1024 + 8 <= kMaxBlocks;
}

gg_fp4_kernel ragged_m_fp4_kernel(const Fp4Params& p, int cus) {
    // Stream or block kernel, in us, at (groups, k, n) x rows a group: (128, 1440, 6344) x 2 115 / 124, (64, 992,
    // 6244) x 2 43 / 49, (128, 2880, 5760) x 1 142 / 151, x 4 211 / 218, x 8 234 / 234, x 16 271 / 250.  With
    // rows of more than 28 KiB a stream workgroup has a CU to itself: (128, 7168, 2048) x 4 183 / 163.
    if (p.m / p.g <= 4 && p.k > 0 && fp4::stream::row_bytes(p) <= fp4::stream::kMaxRowBytes) return GG_FP4_STREAM;
    return p.m > 0 && fp4::tile_ok(p) && fp4::tile_faster(p, cus) ? GG_FP4_TILE : GG_FP4_BLOCK;
}

hipError_t launch_ragged_m_fp4(const Fp4Params& p, int cus, hipStream_t s) {
    switch (ragged_m_fp4_kernel(p, cus)) {
        case GG_FP4_STREAM: return fp4::stream::launch(p, cus, s);
        case GG_FP4_TILE: return fp4::launch_tile(p, cus, s);
        default: return fp4::block::launch(p, cus, s);
    }
}

}  // namespace gg
