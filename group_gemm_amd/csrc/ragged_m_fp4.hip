// ragged_m_fp4.hip -- the MXFP4 non-contracting ragged dot on gfx950: out[r, :] = lhs[r, :] . rhs[h]^T for
// the rows r of group h, both operands e2m1 codes with k contiguous and E8M0 scales in panels
// [ceil(k/256), rows, 8], fp32 accumulation in v_mfma_scale_f32_*_f8f6f4.
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

// scale bytes of k blocks at and past `valid` (of the four in the word) cleared
__device__ inline uint32_t keep_bytes(uint32_t w, int valid) { return valid >= 4 ? w : valid <= 0 ? 0u : w & ((1u << (8 * valid)) - 1u); }

__device__ inline void store1(uint16_t* p, float v) { *p = f32_to_bf16(v); }
__device__ inline void store1(float* p, float v) { *p = v; }

// Four consecutive columns of one row; `left` = columns of the row from here on.
template <typename OutT>
__device__ inline void store4(OutT* o, f32x4 v, int left, bool vec) {
    if (vec && left >= 4) {
        if constexpr (sizeof(OutT) == 2) *(i32x2*)o = i32x2{(int)pack_bf16(v[0], v[1]), (int)pack_bf16(v[2], v[3])};
        else *(f32x4*)o = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) store1(o + e, v[e]);
    }
}

// Split-k kernel: one workgroup makes a tile of 16 MT rows x 16 NT columns, its four waves taking every
// fourth panel of k each and adding their results in LDS.  A wave streams its panels through a private LDS
// ring of D slots (loads straight into LDS, eight rows of 128 bytes an instruction; the waits are on the
// wave's own loads, so the main loop has no barrier), reads the operands back in the instruction's layout
// and multiplies with 16x16x128 instructions, the weights as the first operand so that a lane holds four
// consecutive columns.
template <int MT, int NT, int D>
struct SplitRing {
    static constexpr int X = MT * 16 * kRowBytes, W = NT * 16 * kRowBytes;
    static constexpr int XS = (MT + 1) / 2 * 256, WS = (NT + 1) / 2 * 256;   // 4 bytes a lane and load
    static constexpr int SLOT = X + W + XS + WS;
    static constexpr int LOADS = 2 * MT + 2 * NT + (MT + 1) / 2 + (NT + 1) / 2;
    static constexpr int RED = 4 * MT * NT * 1024;
    static constexpr int BYTES = 4 * D * SLOT > RED ? 4 * D * SLOT : RED;
    static_assert(LOADS * D <= 63, "vmcnt range");
};

template <int MT, int NT, int D, int PER, typename OutT>
__global__ __launch_bounds__(256) void split_kernel(Fp4Params p, int ntiles) {
    using R = SplitRing<MT, NT, D>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[R::BYTES];
    const int t = threadIdx.x, l = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int slot = blockIdx.x / ntiles, col0 = (blockIdx.x % ntiles) * (16 * NT);
    uint32_t flags;
    const RowTile rt = find_row_tile<PER>(p.group_sizes, p.g, p.m, 16 * MT, slot, &flags);
    if (blockIdx.x == 0 && t == 0) *p.status = flags;
    if (rt.grp == -1) return;
    OutT* out = (OutT*)p.out;
    const int cols = min(16 * NT, p.n - col0);
    if (rt.grp == -2) {
        for (int i = t; i < 16 * NT * rt.rows; i += 256) {
            const int r = i / (16 * NT), c = i % (16 * NT);
            if (c < cols) store1(out + (size_t)(rt.row0 + r) * p.n + col0 + c, 0.f);
        }
        return;
    }
    const int rows = rt.rows, panels = (p.k + kPanel - 1) / kPanel, rb = p.k >> 1;
    const i32x4 rx = make_rsrc_v(p.lhs + (size_t)rt.row0 * rb, (uint32_t)rows * (uint32_t)rb);
    const i32x4 rw = make_rsrc_v(p.rhs + ((size_t)rt.grp * p.n + col0) * rb, (uint32_t)cols * (uint32_t)rb);
    const uint8_t* xs0 = p.lhs_scale + (size_t)rt.row0 * 8;
    const uint8_t* ws0 = p.rhs_scale + ((size_t)rt.grp * panels * p.n + col0) * 8;
    const uint32_t ring0 = lds_u32(smem) + (uint32_t)(wave * D * R::SLOT);
    uint8_t* mine = smem + wave * D * R::SLOT;

    // a load brings rows 8 i .. 8 i + 7: lane l row l / 8, into chunk place l % 8
    const int lr = l >> 3;
    auto load = [&](int panel, int s) {
        const uint32_t base = ring0 + (uint32_t)(s * R::SLOT);
        const bool live = panel < panels;
        auto rows_of = [&](i32x4 rsrc, uint32_t at, int count) {
#pragma unroll
            for (int i = 0; i < count; ++i) {
                const int chunk = (l & 7) ^ swizzle(8 * i + lr);
                const uint32_t byte = (uint32_t)panel * kRowBytes + 16u * (uint32_t)chunk;
                const bool ok = live && byte < (uint32_t)rb;
                load_lds16(rsrc, at + 1024u * (uint32_t)i, ok ? (uint32_t)(8 * i + lr) * (uint32_t)rb + byte : kOOB);
            }
        };
        rows_of(rw, base, 2 * NT);
        rows_of(rx, base + R::W, 2 * MT);
        const i32x4 rws = make_rsrc_v(ws0 + (size_t)(live ? panel : 0) * p.n * 8, (uint32_t)cols * 8u);
        const i32x4 rxs = make_rsrc_v(xs0 + (size_t)(live ? panel : 0) * p.m * 8, (uint32_t)rows * 8u);
#pragma unroll
        for (int i = 0; i < (NT + 1) / 2; ++i) load_lds4(rws, base + R::W + R::X + 256u * i, live ? 256u * i + 4u * l : kOOB);
#pragma unroll
        for (int i = 0; i < (MT + 1) / 2; ++i) load_lds4(rxs, base + R::W + R::X + R::WS + 256u * i, live ? 256u * i + 4u * l : kOOB);
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
    for (int s = 0; s < D; ++s) load(wave + 4 * s, s);
    const int r = l & 15, q = l >> 4;
    int s = 0;
    for (int panel = wave; panel < panels; panel += 4) {
        wait_vm<R::LOADS * (D - 1)>();   // the oldest slot is in LDS
        const uint8_t* w = mine + s * R::SLOT;
        const uint8_t* x = w + R::W;
        const uint8_t* ws = x + R::X;
        const uint8_t* xs = ws + R::WS;
        // the lane's k blocks 2 q and 2 q + 1 of the panel: chunks 2 q + h, scale bytes likewise
        i32x4 fw[NT][2], fx[MT][2];
        uint32_t sw[NT], sx[MT];
        const int valid = (p.k >> 5) - panel * 8 - 2 * q;   // blocks of the lane's two that lie inside k
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int row = 16 * j + r;
#pragma unroll
            for (int h = 0; h < 2; ++h) fw[j][h] = *(const i32x4*)(w + row * kRowBytes + (((2 * q + h) ^ swizzle(row)) << 4));
            sw[j] = keep_bytes(*(const uint16_t*)(ws + row * 8 + 2 * q), valid);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = 16 * i + r;
#pragma unroll
            for (int h = 0; h < 2; ++h) fx[i][h] = *(const i32x4*)(x + row * kRowBytes + (((2 * q + h) ^ swizzle(row)) << 4));
            sx[i] = keep_bytes(*(const uint16_t*)(xs + row * 8 + 2 * q), valid);
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);   // the slot has been read (lgkmcnt(0)): it can be filled again
        __builtin_amdgcn_sched_barrier(0);
        load(panel + 4 * D, s);
        s = s + 1 == D ? 0 : s + 1;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(fw[j][0]), widen(fx[i][0]), acc[i][j], kFp4, kFp4, 0, (int)sw[j], 0, (int)sx[i]);
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(fw[j][1]), widen(fx[i][1]), acc[i][j], kFp4, kFp4, 1, (int)sw[j], 1, (int)sx[i]);
            }
    }
    // add the four waves' results (in wave order) and store
    wait_vm<0>();
    __syncthreads();
    f32x4* red = (f32x4*)smem;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) red[((wave * MT + i) * NT + j) * 64 + l] = acc[i][j];
    __syncthreads();
    const bool vec = (p.n & 3) == 0 && ((uintptr_t)p.out & (4 * sizeof(OutT) - 1)) == 0;
    for (int tile = wave; tile < MT * NT; tile += 4) {
        f32x4 v = red[tile * 64 + l];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const f32x4 a = red[(w * MT * NT + tile) * 64 + l];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += a[e];
        }
        const int row = 16 * (tile / NT) + r, col = 16 * (tile % NT) + 4 * q;
        if (row < rows && col < cols) store4(out + (size_t)(rt.row0 + row) * p.n + col0 + col, v, cols - col, vec);
    }
}

template <int MT, int NT, int D, int PER>
hipError_t launch_split_per(const Fp4Params& p, int64_t grid, int ntiles, hipStream_t s) {
    if (p.out_f32) hipLaunchKernelGGL((split_kernel<MT, NT, D, PER, float>), dim3((uint32_t)grid), dim3(256), 0, s, p, ntiles);
    else hipLaunchKernelGGL((split_kernel<MT, NT, D, PER, uint16_t>), dim3((uint32_t)grid), dim3(256), 0, s, p, ntiles);
    return hipGetLastError();
}

// row tiles (and tiles of rows past the total) that any group_sizes can give
inline int64_t slot_bound(const Fp4Params& p, int tile_rows) { return (p.g < p.m ? p.g : p.m) + (int64_t)p.m / tile_rows + 1; }

template <int MT, int NT, int D>
hipError_t launch_split(const Fp4Params& p, hipStream_t s) {
    const int ntiles = (p.n + 16 * NT - 1) / (16 * NT);
    const int64_t grid = slot_bound(p, 16 * MT) * (ntiles > 0 ? ntiles : 1);
    const int nt = ntiles > 0 ? ntiles : 1;
    if (p.g <= 64) return launch_split_per<MT, NT, D, 1>(p, grid, nt, s);
    if (p.g <= 256) return launch_split_per<MT, NT, D, 4>(p, grid, nt, s);
    return launch_split_per<MT, NT, D, 16>(p, grid, nt, s);
}

}  // namespace fp4

bool ragged_m_fp4_grid_ok(const Fp4Params& p) {
    // (column indices past n must not leave 32 bits either)
    return p.n <= INT32_MAX - 256 && fp4::slot_bound(p, 16) * ((p.n + 15) / 16) <= INT32_MAX && (int64_t)64 * (p.k >> 1) < (int64_t(1) << 31);
}

hipError_t launch_ragged_m_fp4(const Fp4Params& p, int cus, hipStream_t s) {
    (void)cus;
    const int64_t per = p.m / p.g;
    if (per <= 4) return fp4::launch_split<1, 1, 4>(p, s);
    return fp4::launch_split<2, 2, 2>(p, s);
}

}  // namespace gg
