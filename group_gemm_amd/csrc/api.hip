// api.hip -- the C ABI: argument validation, workspace layout, grid sizing and launches.
// Host code only; it never reads group_sizes or any other device data (except in
// gg_read_device_status, which exists for tests), never synchronises and never allocates,
// so every call can be captured in a HIP graph.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "groupgemm.h"
#include "launch.hpp"

// Scratch of ragged_dot_m_noalloc: the per-call state that the workspace holds for the other
// calls (status word at offset 0, the 8 tile-queue counters at offset 64), kept in a
// file-scope device array for callers that cannot allocate.  Each GPU holds its own copy
// for the life of the process; every no-allocation call on a GPU shares it.
constexpr size_t kScratchBytes = 256;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

namespace {

constexpr size_t kHeader = 256;   // workspace bytes before any padded buffer (status word first)
constexpr int64_t kMaxCopies = int64_t(1) << 30;   // moe_permute: tokens * top_k
constexpr size_t kQueueOffset = 64;                 // workspace header bytes before the 8 tile queues

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

size_t elem_bytes(gg_dtype d) { return d == GG_DT_F32 ? 4 : d == GG_DT_BF16 ? 2 : 1; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// whether two arrays share a byte (sizes are at most 2^63 and addresses below 2^48: no sum wraps)
bool overlap(const void* a, uint64_t an, const void* b, uint64_t bn) {
    const uint64_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return an > 0 && bn > 0 && a0 < b0 + bn && b0 < a0 + an;
}

// Compute units of the current device, cached per device.
int device_cus(int* cus) {
    static int cache[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return -1;
    if (dev >= 0 && dev < 64 && cache[dev] > 0) { *cus = cache[dev]; return 0; }
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) return -1;
    if (dev >= 0 && dev < 64) cache[dev] = v;
    *cus = v;
    return 0;
}

// Persistent grid: one workgroup per CU (the big-tile kernels hold 128+ KiB of LDS),
// never more than there are tiles, at least 1 so the status word is always written.
int persistent_grid(int64_t tile_bound, int per_cu, int cus) {
    int64_t g = (int64_t)cus * per_cu;
    if (tile_bound < g) g = tile_bound;
    if (g < 1) g = 1;
    return (int)g;
}

// Launchers return hipErrorInvalidConfiguration for more workgroups than a launch holds.
gg_status launched(hipError_t e) {
    return e == hipSuccess ? GG_OK : e == hipErrorInvalidConfiguration ? GG_ERR_BAD_SHAPE : GG_ERR_HIP;
}

bool fits_i32(int64_t x) { return x >= 0 && x <= INT32_MAX; }

// whether two matrices share a byte: rows of `width` bytes, `pitch` apart (rows of one pitch may interleave)
struct Span { const void* p; uint64_t rows, width, pitch; };
bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
    if (!overlap(a.p, (a.rows - 1) * a.pitch + a.width, b.p, (b.rows - 1) * b.pitch + b.width)) return false;
    if (a.pitch != b.pitch || a.rows == 1 || b.rows == 1) return true;
    const uint64_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const uint64_t d = b0 >= a0 ? (b0 - a0) % a.pitch : (a.pitch - (a0 - b0) % a.pitch) % a.pitch;   // columns that b begins after a
    return d < a.width || d + b.width > a.pitch;
}
Span dense(const void* p, uint64_t bytes) { return {p, 1, bytes, bytes}; }
// whether `out` shares a byte with any of `others`
template <typename... S> bool meets(const Span& out, const S&... others) { return (overlap(out, others) || ...); }

// Shape and group-size checks shared by every entry point.
gg_status check_shape(int64_t m, int64_t k, int64_t n, int32_t g, const int32_t* gs) {
    if (!gs) return GG_ERR_NULL_PTR;
    if (m < 0 || k < 0 || n < 0 || g < 1 || g > GG_MAX_GROUPS) return GG_ERR_BAD_SHAPE;
    if (!fits_i32(m) || !fits_i32(k) || !fits_i32(n)) return GG_ERR_BAD_SHAPE;
    if (!aligned(gs, 4)) return GG_ERR_MISALIGNED;
    return GG_OK;
}

gg_status check_common(int64_t m, int64_t k, int64_t n, int32_t g, const int32_t* gs, void* ws, size_t ws_bytes,
                       size_t need) {
    if (!gs || !ws) return GG_ERR_NULL_PTR;
    gg_status st = check_shape(m, k, n, g, gs);
    if (st != GG_OK) return st;
    if (!aligned(ws, 16)) return GG_ERR_MISALIGNED;
    if (ws_bytes < need) return GG_ERR_WORKSPACE_TOO_SMALL;
    return GG_OK;
}

// ragged_dot_m body, shared with the batched stage of padded_dot (uniform_rows > 0).
// Epilogue of the ring kernels: out = alpha * acc + bias[h] + beta * out.  `on` false: plain
// store (every kernel family); true: only the ring kernels implement it.
struct EpiArgs {
    bool on = false;
    const float* bias = nullptr;
    int64_t bias_stride = 0;
    float alpha = 1.f, beta = 0.f;
};

// `status` may be NULL (the padded form's batched stage leaves the word to the scatter);
// `ws` is the caller's workspace, whose header also holds the bf16 kernel's tile queues.
gg_status run_m(const void* lhs, const void* rhs, const int32_t* gs, void* out, int64_t m, int64_t k, int64_t n,
                int32_t g, gg_dtype in, gg_dtype outd, const uint8_t* ls, const uint8_t* rs, uint32_t* status,
                void* ws, int uniform_rows, hipStream_t s, bool rhs_nk = false, const EpiArgs& ep = EpiArgs()) {
    int cus;
    if (device_cus(&cus) != 0) return GG_ERR_HIP;
    gg::MParams p{};
    p.lhs = lhs; p.rhs = rhs; p.lhs_scale = ls; p.rhs_scale = rs; p.group_sizes = gs; p.out = out; p.status = status;
    p.m = (int)m; p.k = (int)k; p.n = (int)n; p.g = g; p.uniform_rows = uniform_rows;
    p.out_f32 = outd == GG_DT_F32;
    p.rhs_nk = rhs_nk ? 1 : 0;
    p.epi = ep.on ? 1 : 0; p.bias = ep.bias; p.bias_stride = ep.bias_stride; p.alpha = ep.alpha; p.beta = ep.beta;
    p.tile_queue = (int*)((char*)ws + kQueueOffset);
    hipError_t e;
    if (rhs_nk) {   // [g,n,k] weights: the bf16 ring kernel only
        const bool vec = aligned(lhs, 16) && aligned(rhs, 16) && aligned(out, 16) && k % 8 == 0 && n % 8 == 0;
        if (in != GG_DT_BF16 || !vec || !gg::ragged_m_bf16_fast_ok(p)) return GG_ERR_UNSUPPORTED;
        int64_t bound = (cdiv64(m, gg::ragged_m_bf16_fast_bm(p)) + g + 1) * cdiv64(n, 256);
        if (!fits_i32(bound)) return GG_ERR_BAD_SHAPE;
        e = gg::launch_ragged_m_bf16_fast(p, persistent_grid(bound, 1, cus), s);
    } else if (in == GG_DT_F32) {
        if (ep.on) return GG_ERR_UNSUPPORTED;
        gg::TileShape ts = gg::tiles_m_f32();
        int64_t bound = (cdiv64(m, ts.bm) + g + 1) * cdiv64(n, ts.bn);
        if (!fits_i32(bound)) return GG_ERR_BAD_SHAPE;
        e = gg::launch_ragged_m_f32(p, persistent_grid(bound, 4, cus), s);
    } else if (in == GG_DT_BF16) {
        const bool vec = aligned(lhs, 16) && aligned(rhs, 16) && aligned(out, 16) && k % 8 == 0 && n % 8 == 0;
        const bool fast = vec && gg::ragged_m_bf16_fast_ok(p);
        gg::TileShape ts = gg::tiles_m_bf16();
        if (fast) ts = {gg::ragged_m_bf16_fast_bm(p), 256};
        int64_t bound = (cdiv64(m, ts.bm) + g + 1) * cdiv64(n, ts.bn);
        if (!fits_i32(bound)) return GG_ERR_BAD_SHAPE;
        if (ep.on && !fast) return GG_ERR_UNSUPPORTED;
        if (fast) e = gg::launch_ragged_m_bf16_fast(p, persistent_grid(bound, 1, cus), s);
        else e = gg::launch_ragged_m_bf16(p, persistent_grid(bound, 1, cus), vec, s);
    } else {
        const bool fast = aligned(lhs, 16) && aligned(rhs, 16) && aligned(out, 16) && aligned(ls, 4) && aligned(rs, 4) &&
                          gg::ragged_m_mx_fast_ok(p);
        gg::TileShape ts = gg::tiles_m_e4m3();
        if (fast) ts = {256, 256};
        int64_t bound = (cdiv64(m, ts.bm) + g + 1) * cdiv64(n, ts.bn);
        if (!fits_i32(bound)) return GG_ERR_BAD_SHAPE;
        if (ep.on && !fast) return GG_ERR_UNSUPPORTED;
        if (fast) e = gg::launch_ragged_m_mx_fast(p, persistent_grid(bound, 1, cus), s);
        else e = gg::launch_ragged_m_e4m3(p, persistent_grid(bound, 1, cus), s);
    }
    return e == hipSuccess ? GG_OK : GG_ERR_HIP;
}

gg_status run_k(const void* lhs, const void* dout, const int32_t* gs, void* out, int64_t m, int64_t k, int64_t n,
                int32_t g, gg_dtype in, gg_dtype outd, uint32_t* status, int uniform_rows, hipStream_t s,
                const EpiArgs& ep = EpiArgs()) {
    int cus;
    if (device_cus(&cus) != 0) return GG_ERR_HIP;
    gg::KParams p{};
    p.lhs = lhs; p.dout = dout; p.group_sizes = gs; p.out = out; p.status = status;
    p.m = (int)m; p.k = (int)k; p.n = (int)n; p.g = g; p.uniform_rows = uniform_rows;
    p.out_f32 = outd == GG_DT_F32;
    p.epi = ep.on ? 1 : 0; p.alpha = ep.alpha; p.beta = ep.beta;
    hipError_t e;
    if (in == GG_DT_F32) {
        if (ep.on) return GG_ERR_UNSUPPORTED;
        gg::TileShape ts = gg::tiles_k_f32();
        int64_t bound = (int64_t)g * cdiv64(k, ts.bm) * cdiv64(n, ts.bn);
        if (!fits_i32(bound)) return GG_ERR_BAD_SHAPE;
        e = gg::launch_ragged_k_f32(p, persistent_grid(bound, 4, cus), s);
    } else {
        gg::TileShape ts = gg::tiles_k_bf16();
        int64_t bound = (int64_t)g * cdiv64(k, ts.bm) * cdiv64(n, ts.bn);
        if (!fits_i32(bound)) return GG_ERR_BAD_SHAPE;
        const bool vec = aligned(lhs, 16) && aligned(dout, 16) && k % 8 == 0 && n % 8 == 0;
        const bool fast = vec && aligned(out, 16) && gg::ragged_k_bf16_fast_ok(p);
        if (ep.on && !fast) return GG_ERR_UNSUPPORTED;
        if (fast) e = gg::launch_ragged_k_bf16_fast(p, persistent_grid(bound, 1, cus), s);
        else e = gg::launch_ragged_k_bf16(p, persistent_grid(bound, 1, cus), vec, s);
    }
    return e == hipSuccess ? GG_OK : GG_ERR_HIP;
}

// Device address of `scratch` on the current device, resolved once per device with that
// device current (host code must never pass the array's own name: that is a host-side
// stand-in, not a device address).  NULL if the lookup fails.
void* scratch_address() {
    static std::mutex mu;
    static void* addr[64] = {nullptr};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess) return nullptr;
        addr[dev] = p;
    }
    return addr[dev];
}

// Workspace of ragged_lora_grad behind the header: offsets of its parts.
struct LoraGradLayout { size_t bt, at, t, u, parts, bytes; };
LoraGradLayout lora_grad_layout(int64_t m, int64_t k, int64_t n, int r, int32_t g, gg_dtype dtype) {
    const size_t es = elem_bytes(dtype), rows = align_up((size_t)m * r * 4, 256);
    const int splits = gg::lora_splits(m, n, r, g);
    const int64_t chunk = gg::lora_chunk(m, k, n);
    LoraGradLayout w{};
    w.bt = 0;
    w.at = w.bt + align_up((size_t)g * n * r * es, 256);
    w.u = w.at + align_up((size_t)g * k * r * es, 256);
    w.t = splits > 1 ? w.u + rows : w.u;
    w.parts = w.t + (size_t)splits * rows;
    w.bytes = w.parts + align_up(2 * (size_t)cdiv64(m, chunk) * (size_t)(k + n) * r * 4, 256);
    return w;
}

// [rows, k] in eights of a row's elements, with k % 8 checked elsewhere
bool eights_ok(int64_t rows, int64_t k) {
    return fits_i32(rows) && fits_i32(k) && (k == 0 || rows <= ((int64_t(1) << 34) - 8) / k);
}

bool floats(gg_dtype d) { return d == GG_DT_F32 || d == GG_DT_BF16; }

bool m_dtypes_ok(gg_dtype in, gg_dtype out) {
    if (in == GG_DT_F32) return out == GG_DT_F32;
    if (in == GG_DT_BF16 || in == GG_DT_E4M3) return out == GG_DT_BF16 || out == GG_DT_F32;
    return false;
}
bool k_dtypes_ok(gg_dtype in, gg_dtype out) {
    if (in == GG_DT_F32) return out == GG_DT_F32;
    if (in == GG_DT_BF16) return out == GG_DT_F32 || out == GG_DT_BF16;
    return false;
}

}  // namespace

extern "C" {

int gg_abi_version(void) { return GG_ABI_VERSION; }

const char* gg_status_string(gg_status s) {
    switch (s) {
        case GG_OK: return "ok";
        case GG_ERR_NULL_PTR: return "a required pointer is NULL";
        case GG_ERR_BAD_SHAPE: return "bad shape (negative size, g outside [1, GG_MAX_GROUPS], or too large)";
        case GG_ERR_BAD_DTYPE: return "unsupported element type combination";
        case GG_ERR_MISALIGNED: return "misaligned pointer";
        case GG_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
        case GG_ERR_UNSUPPORTED: return "unsupported argument combination";
        case GG_ERR_HIP: return "HIP runtime error";
        default: break;
    }
    return "unknown status";
}

size_t gg_workspace_bytes(gg_op op, int64_t m, int64_t k, int64_t n, int32_t g, int64_t capacity, gg_dtype in) {
    if (m < 0 || k < 0 || n < 0 || g < 1 || g > GG_MAX_GROUPS) return 0;
    if (in != GG_DT_F32 && in != GG_DT_BF16 && in != GG_DT_E4M3 &&
        !(in == GG_DT_E2M1 && (op == GG_OP_RAGGED_M || op == GG_OP_PERMUTE)))
        return 0;
    switch (op) {
        case GG_OP_RAGGED_M: return kHeader;
        case GG_OP_RAGGED_K: {
            if (in != GG_DT_E4M3 || !fits_i32(m) || !fits_i32(k) || !fits_i32(n)) return kHeader;
            const int splits = gg::ragged_k_mx_splits(m, k, n, g);
            return kHeader + (splits > 1 ? (size_t)g * splits * (size_t)k * (size_t)n * 4 : 0);
        }
        case GG_OP_PADDED_M: {
            if (capacity < 1) return 0;
            const size_t rows = (size_t)g * (size_t)capacity;
            size_t b = kHeader;
            b += align_up(rows * (size_t)k * elem_bytes(in), 256);    // padded lhs
            b += align_up(rows * (size_t)n * 4, 256);                 // padded result (room for fp32)
            if (in == GG_DT_E4M3) b += align_up(rows * (size_t)(k / 32), 256);   // padded lhs scales
            return b;
        }
        case GG_OP_PADDED_K: {
            if (capacity < 1) return 0;
            const size_t rows = (size_t)g * (size_t)capacity;
            return kHeader + align_up(rows * (size_t)k * elem_bytes(in), 256) + align_up(rows * (size_t)n * elem_bytes(in), 256);
        }
        case GG_OP_PERMUTE: {
            if (m > kMaxCopies) return 0;
            const gg::PermuteGeometry pg = gg::permute_geometry(m);
            return kHeader + align_up((size_t)pg.nblk * (size_t)g * 4, 256) + align_up((size_t)pg.nblk * 4, 256);
        }
        case GG_OP_LORA: {   // capacity: r
            if (capacity < 1 || capacity > GG_MAX_RANK || !fits_i32(m) || !fits_i32(k) || in == GG_DT_E4M3) return 0;
            return kHeader + align_up((size_t)gg::lora_splits(m, k, (int)capacity, g) * (size_t)m * (size_t)capacity * 4, 256);
        }
        case GG_OP_LORA_GRAD: {
            if (capacity < 1 || capacity > GG_MAX_RANK || !fits_i32(m) || !fits_i32(k) || !fits_i32(n) || in == GG_DT_E4M3) return 0;
            if (!gg::lora_grad_grid_ok(m, k, n, g)) return 0;   // (and the sizes below stay within 64 bits)
            return kHeader + lora_grad_layout(m, k, n, (int)capacity, g, in).bytes;
        }
        default: break;
    }
    return 0;
}

gg_status ragged_dot_m(const void* lhs, const void* rhs, const int32_t* group_sizes, void* out, int64_t m, int64_t k,
                       int64_t n, int32_t g, gg_dtype in_dtype, gg_dtype out_dtype, const uint8_t* lhs_scale,
                       const uint8_t* rhs_scale, void* workspace, size_t workspace_bytes, void* stream) {
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes, kHeader);
    if (st != GG_OK) return st;
    if (!m_dtypes_ok(in_dtype, out_dtype)) return GG_ERR_BAD_DTYPE;
    if ((m * k > 0 && !lhs) || (k * n > 0 && !rhs) || (m * n > 0 && !out)) return GG_ERR_NULL_PTR;
    const size_t es = elem_bytes(in_dtype);
    if (!aligned(lhs, es) || !aligned(rhs, es) || !aligned(out, elem_bytes(out_dtype))) return GG_ERR_MISALIGNED;
    if (in_dtype == GG_DT_E4M3) {
        if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
        if ((m * k > 0 && !lhs_scale) || (k * n > 0 && !rhs_scale)) return GG_ERR_NULL_PTR;
        if (!aligned(lhs, 16) || !aligned(rhs, 16)) return GG_ERR_MISALIGNED;
    }
    return run_m(lhs, rhs, group_sizes, out, m, k, n, g, in_dtype, out_dtype, lhs_scale, rhs_scale, (uint32_t*)workspace, workspace,
                 0, (hipStream_t)stream);
}

gg_status ragged_dot_m_noalloc(const void* lhs, const void* rhs, const int32_t* group_sizes, void* out, int64_t m,
                               int64_t k, int64_t n, int32_t g, gg_dtype in_dtype, gg_dtype out_dtype,
                               const uint8_t* lhs_scale, const uint8_t* rhs_scale, uint32_t* status, void* stream) {
    // the scratch must hold what the workspace of ragged_dot_m would (the same for any shape)
    const size_t need = gg_workspace_bytes(GG_OP_RAGGED_M, m, k, n, g, 0, in_dtype);
    if (need > kScratchBytes) return GG_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(status, 4)) return GG_ERR_MISALIGNED;
    gg_status st = check_shape(m, k, n, g, group_sizes);
    if (st != GG_OK) return st;
    if (!m_dtypes_ok(in_dtype, out_dtype)) return GG_ERR_BAD_DTYPE;
    if ((m * k > 0 && !lhs) || (k * n > 0 && !rhs) || (m * n > 0 && !out)) return GG_ERR_NULL_PTR;
    const size_t es = elem_bytes(in_dtype);
    if (!aligned(lhs, es) || !aligned(rhs, es) || !aligned(out, elem_bytes(out_dtype))) return GG_ERR_MISALIGNED;
    if (in_dtype == GG_DT_E4M3) {
        if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
        if ((m * k > 0 && !lhs_scale) || (k * n > 0 && !rhs_scale)) return GG_ERR_NULL_PTR;
        if (!aligned(lhs, 16) || !aligned(rhs, 16)) return GG_ERR_MISALIGNED;
    }
    void* ws = scratch_address();   // looked up only once every argument has passed its check
    if (!ws) return GG_ERR_HIP;
    return run_m(lhs, rhs, group_sizes, out, m, k, n, g, in_dtype, out_dtype, lhs_scale, rhs_scale,
                 status ? status : (uint32_t*)ws, ws, 0, (hipStream_t)stream);
}

gg_status ragged_dot_m_nk(const void* lhs, const void* rhs_nk, const int32_t* group_sizes, void* out, int64_t m,
                          int64_t k, int64_t n, int32_t g, gg_dtype in_dtype, gg_dtype out_dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes, kHeader);
    if (st != GG_OK) return st;
    if (in_dtype != GG_DT_BF16) return GG_ERR_UNSUPPORTED;
    if (!m_dtypes_ok(in_dtype, out_dtype)) return GG_ERR_BAD_DTYPE;
    if ((m * k > 0 && !lhs) || (k * n > 0 && !rhs_nk) || (m * n > 0 && !out)) return GG_ERR_NULL_PTR;
    if (!aligned(lhs, 16) || !aligned(rhs_nk, 16) || !aligned(out, 16)) return GG_ERR_MISALIGNED;
    if (k % 8 != 0 || n % 8 != 0) return GG_ERR_UNSUPPORTED;
    return run_m(lhs, rhs_nk, group_sizes, out, m, k, n, g, in_dtype, out_dtype, nullptr, nullptr, (uint32_t*)workspace, workspace,
                 0, (hipStream_t)stream, true);
}

gg_status ragged_dot_m_epilogue(const void* lhs, const void* rhs, const int32_t* group_sizes, void* out, int64_t m,
                                int64_t k, int64_t n, int32_t g, gg_dtype in_dtype, gg_dtype out_dtype,
                                const uint8_t* lhs_scale, const uint8_t* rhs_scale, const float* bias, int64_t bias_stride,
                                float alpha, float beta, void* workspace, size_t workspace_bytes, void* stream) {
    if (bias && (bias_stride < n || !aligned(bias, 4))) return bias_stride < n ? GG_ERR_BAD_SHAPE : GG_ERR_MISALIGNED;
    EpiArgs ep;
    ep.on = bias != nullptr || alpha != 1.f || beta != 0.f;
    ep.bias = bias; ep.bias_stride = bias_stride; ep.alpha = alpha; ep.beta = beta;
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes, kHeader);
    if (st != GG_OK) return st;
    if (!m_dtypes_ok(in_dtype, out_dtype)) return GG_ERR_BAD_DTYPE;
    if ((m * k > 0 && !lhs) || (k * n > 0 && !rhs) || (m * n > 0 && !out)) return GG_ERR_NULL_PTR;
    const size_t es = elem_bytes(in_dtype);
    if (!aligned(lhs, es) || !aligned(rhs, es) || !aligned(out, elem_bytes(out_dtype))) return GG_ERR_MISALIGNED;
    if (in_dtype == GG_DT_E4M3) {
        if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
        if ((m * k > 0 && !lhs_scale) || (k * n > 0 && !rhs_scale)) return GG_ERR_NULL_PTR;
        if (!aligned(lhs, 16) || !aligned(rhs, 16)) return GG_ERR_MISALIGNED;
    }
    return run_m(lhs, rhs, group_sizes, out, m, k, n, g, in_dtype, out_dtype, lhs_scale, rhs_scale, (uint32_t*)workspace, workspace,
                 0, (hipStream_t)stream, false, ep);
}

gg_status ragged_dot_k_epilogue(const void* lhs, const void* dout, const int32_t* group_sizes, void* out, int64_t m,
                                int64_t k, int64_t n, int32_t g, gg_dtype in_dtype, gg_dtype out_dtype, float alpha,
                                float beta, void* workspace, size_t workspace_bytes, void* stream) {
    EpiArgs ep;
    ep.on = alpha != 1.f || beta != 0.f;
    ep.alpha = alpha; ep.beta = beta;
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes, kHeader);
    if (st != GG_OK) return st;
    if (!k_dtypes_ok(in_dtype, out_dtype)) return GG_ERR_BAD_DTYPE;
    if ((m * k > 0 && !lhs) || (m * n > 0 && !dout) || (k * n > 0 && !out)) return GG_ERR_NULL_PTR;
    const size_t es = elem_bytes(in_dtype);
    if (!aligned(lhs, es) || !aligned(dout, es) || !aligned(out, elem_bytes(out_dtype))) return GG_ERR_MISALIGNED;
    return run_k(lhs, dout, group_sizes, out, m, k, n, g, in_dtype, out_dtype, (uint32_t*)workspace, 0,
                 (hipStream_t)stream, ep);
}

gg_status ragged_dot_m_gated(const void* lhs, const void* w0, const void* w1, const int32_t* group_sizes, void* out,
                             int64_t m, int64_t k, int64_t n, int32_t g, gg_dtype in_dtype, gg_dtype out_dtype,
                             gg_activation act, const float* bias0, const float* bias1, int64_t bias_stride,
                             void* workspace, size_t workspace_bytes, void* stream) {
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes, kHeader);
    if (st != GG_OK) return st;
    if (in_dtype != GG_DT_BF16) return GG_ERR_UNSUPPORTED;
    if (!m_dtypes_ok(in_dtype, out_dtype)) return GG_ERR_BAD_DTYPE;
    if (act != GG_ACT_SILU && act != GG_ACT_GELU_TANH) return GG_ERR_UNSUPPORTED;
    if ((m * k > 0 && !lhs) || (k * n > 0 && (!w0 || !w1)) || (m * n > 0 && !out)) return GG_ERR_NULL_PTR;
    if ((bias0 || bias1) && bias_stride < n) return GG_ERR_BAD_SHAPE;
    if (!aligned(bias0, 4) || !aligned(bias1, 4)) return GG_ERR_MISALIGNED;
    if (!aligned(lhs, 16) || !aligned(w0, 16) || !aligned(w1, 16) || !aligned(out, 16)) return GG_ERR_MISALIGNED;
    if (k % 8 != 0 || n % 8 != 0) return GG_ERR_UNSUPPORTED;
    int cus;
    if (device_cus(&cus) != 0) return GG_ERR_HIP;
    gg::GParams p{};
    p.lhs = lhs; p.w0 = w0; p.w1 = w1; p.group_sizes = group_sizes; p.out = out; p.status = (uint32_t*)workspace;
    p.bias0 = bias0; p.bias1 = bias1; p.bias_stride = bias_stride;
    p.m = (int)m; p.k = (int)k; p.n = (int)n; p.g = g; p.out_f32 = out_dtype == GG_DT_F32; p.act = (int)act;
    if (!gg::ragged_m_gated_ok(p)) return GG_ERR_UNSUPPORTED;
    const int64_t bound = (cdiv64(m, 256) + g + 1) * cdiv64(n, 128);
    if (!fits_i32(bound)) return GG_ERR_BAD_SHAPE;
    return gg::launch_ragged_m_gated(p, persistent_grid(bound, 1, cus), (hipStream_t)stream) == hipSuccess ? GG_OK
                                                                                                           : GG_ERR_HIP;
}

gg_status ragged_dot_k(const void* lhs, const void* dout, const int32_t* group_sizes, void* out, int64_t m, int64_t k,
                       int64_t n, int32_t g, gg_dtype in_dtype, gg_dtype out_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes, kHeader);
    if (st != GG_OK) return st;
    if (!k_dtypes_ok(in_dtype, out_dtype)) return GG_ERR_BAD_DTYPE;
    if ((m * k > 0 && !lhs) || (m * n > 0 && !dout) || (k * n > 0 && !out)) return GG_ERR_NULL_PTR;
    const size_t es = elem_bytes(in_dtype);
    if (!aligned(lhs, es) || !aligned(dout, es) || !aligned(out, elem_bytes(out_dtype))) return GG_ERR_MISALIGNED;
    return run_k(lhs, dout, group_sizes, out, m, k, n, g, in_dtype, out_dtype, (uint32_t*)workspace, 0,
                 (hipStream_t)stream);
}

gg_status padded_dot(gg_op mode, const void* a, const void* b, const int32_t* group_sizes, void* out, int64_t m,
                     int64_t k, int64_t n, int32_t g, int64_t capacity, gg_dtype in_dtype, gg_dtype out_dtype,
                     const uint8_t* a_scale, const uint8_t* b_scale, void* workspace, size_t workspace_bytes,
                     void* stream) {
    if (mode != GG_OP_PADDED_M && mode != GG_OP_PADDED_K) return GG_ERR_UNSUPPORTED;
    if (capacity < 1 || !fits_i32(capacity) || !fits_i32((int64_t)g * capacity)) return GG_ERR_BAD_SHAPE;
    const size_t need = gg_workspace_bytes(mode, m, k, n, g, capacity, in_dtype);
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes, need ? need : kHeader);
    if (st != GG_OK) return st;
    const bool is_m = mode == GG_OP_PADDED_M;
    if (is_m ? !m_dtypes_ok(in_dtype, out_dtype) : !k_dtypes_ok(in_dtype, out_dtype)) return GG_ERR_BAD_DTYPE;
    if (need == 0) return GG_ERR_BAD_SHAPE;
    const size_t es = elem_bytes(in_dtype), os = elem_bytes(out_dtype);
    if (!a || !b || !out) return GG_ERR_NULL_PTR;
    if (!aligned(a, es) || !aligned(b, es) || !aligned(out, os)) return GG_ERR_MISALIGNED;
    if (in_dtype == GG_DT_E4M3) {
        if (!is_m) return GG_ERR_BAD_DTYPE;
        if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
        if (!a_scale || !b_scale) return GG_ERR_NULL_PTR;
        if (!aligned(a, 16) || !aligned(b, 16)) return GG_ERR_MISALIGNED;
    }
    hipStream_t s = (hipStream_t)stream;
    uint32_t* status = (uint32_t*)workspace;
    uint8_t* base = (uint8_t*)workspace + kHeader;
    const int64_t rows = (int64_t)g * capacity;
    uint8_t* pa = base;
    uint8_t* pb = pa + align_up((size_t)rows * (size_t)k * es, 256);
    hipError_t e;
    if (is_m) {
        // 1. expand: lhs rows -> [g, C, k] (+ their scales)
        e = gg::launch_pad_scatter(a, pa, group_sizes, (int)m, g, (int)capacity, (long long)k * (long long)es, status, s);
        if (e != hipSuccess) return GG_ERR_HIP;
        uint8_t* psc = pb + align_up((size_t)rows * (size_t)n * 4, 256);
        if (in_dtype == GG_DT_E4M3) {
            e = gg::launch_pad_scatter(a_scale, psc, group_sizes, (int)m, g, (int)capacity, (long long)(k / 32), nullptr, s);
            if (e != hipSuccess) return GG_ERR_HIP;
        }
        // 2. one uniform batched GEMM [g, C, k] x [g, k, n] -> [g, C, n]
        st = run_m(pa, b, group_sizes, pb, rows, k, n, g, in_dtype, out_dtype, psc, b_scale, nullptr, workspace, (int)capacity, s);
        if (st != GG_OK) return st;
        // 3. compact: [g, C, n] -> [m, n]
        e = gg::launch_pad_gather(pb, out, group_sizes, (int)m, g, (int)capacity, (long long)n * (long long)os, s);
        return e == hipSuccess ? GG_OK : GG_ERR_HIP;
    }
    // contracting form: expand both operands, then one uniform batched contraction
    e = gg::launch_pad_scatter(a, pa, group_sizes, (int)m, g, (int)capacity, (long long)k * (long long)es, status, s);
    if (e != hipSuccess) return GG_ERR_HIP;
    e = gg::launch_pad_scatter(b, pb, group_sizes, (int)m, g, (int)capacity, (long long)n * (long long)es, nullptr, s);
    if (e != hipSuccess) return GG_ERR_HIP;
    return run_k(pa, pb, group_sizes, out, rows, k, n, g, in_dtype, out_dtype, nullptr, (int)capacity, s);
}

gg_status moe_permute(const void* x, const uint8_t* x_scale, const int32_t* experts, void* sorted_x,
                      uint8_t* sorted_scale, int32_t* group_sizes, int32_t* sorted_to_copy, int32_t* copy_to_sorted,
                      int64_t tokens, int32_t top_k, int64_t k, int32_t g, gg_dtype dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
    if (!group_sizes || !workspace) return GG_ERR_NULL_PTR;
    if (tokens < 0 || top_k < 1 || k < 0 || g < 1 || g > GG_MAX_GROUPS || !fits_i32(k)) return GG_ERR_BAD_SHAPE;
    if (tokens > kMaxCopies / top_k) return GG_ERR_BAD_SHAPE;
    if (dtype != GG_DT_F32 && dtype != GG_DT_BF16 && dtype != GG_DT_E4M3 && dtype != GG_DT_E2M1) return GG_ERR_BAD_DTYPE;
    const int64_t M = tokens * top_k;
    if (M > 0 && (!experts || !sorted_to_copy || !copy_to_sorted)) return GG_ERR_NULL_PTR;
    if (tokens * k > 0 && (!x || !sorted_x)) return GG_ERR_NULL_PTR;
    const bool fp4 = dtype == GG_DT_E2M1, mx = dtype == GG_DT_E4M3 || fp4;
    if (mx && k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if (mx && tokens * k > 0 && (!x_scale || !sorted_scale)) return GG_ERR_NULL_PTR;
    if (!mx && (x_scale || sorted_scale)) return GG_ERR_BAD_DTYPE;
    const size_t es = elem_bytes(dtype);
    if (!aligned(x, es) || !aligned(sorted_x, es) || !aligned(experts, 4) || !aligned(group_sizes, 4) ||
        !aligned(sorted_to_copy, 4) || !aligned(copy_to_sorted, 4) || !aligned(workspace, 16))
        return GG_ERR_MISALIGNED;
    if (fp4 && (!aligned(x_scale, 8) || !aligned(sorted_scale, 8))) return GG_ERR_MISALIGNED;
    if (fp4 && cdiv64(k, 256) > 65535) return GG_ERR_BAD_SHAPE;
    if (workspace_bytes < gg_workspace_bytes(GG_OP_PERMUTE, M, k, 0, g, 0, dtype)) return GG_ERR_WORKSPACE_TOO_SMALL;
    const gg::PermuteGeometry pg = gg::permute_geometry(M);
    uint8_t* ws = (uint8_t*)workspace;
    gg::PermuteArgs a{};
    a.x = x; a.x_scale = mx ? x_scale : nullptr; a.experts = experts;
    a.sorted_x = sorted_x; a.sorted_scale = mx ? sorted_scale : nullptr;
    a.group_sizes = group_sizes; a.sorted_to_copy = sorted_to_copy; a.copy_to_sorted = copy_to_sorted;
    a.status = (uint32_t*)ws;
    a.total_routed = (int*)(ws + 4);
    a.counts = (int*)(ws + kHeader);
    a.bad = (int*)(ws + kHeader + align_up((size_t)pg.nblk * (size_t)g * 4, 256));
    a.tokens = (int)tokens; a.top_k = top_k; a.g = g;
    a.row_bytes = fp4 ? k / 2 : k * (int64_t)es;
    a.scale_row_bytes = mx && !fp4 ? k / 32 : 0;
    a.scale_panels = fp4 ? (int)cdiv64(k, 256) : 0;
    return launched(gg::launch_permute(a, (hipStream_t)stream));
}

gg_status moe_unpermute(const void* y, const int32_t* copy_to_sorted, const float* weights, void* out, int64_t tokens,
                        int32_t top_k, int64_t n, gg_dtype in_dtype, gg_dtype out_dtype, void* stream) {
    if (tokens < 0 || top_k < 1 || n < 0 || !fits_i32(n)) return GG_ERR_BAD_SHAPE;
    if (tokens > 0 && (!copy_to_sorted || !weights)) return GG_ERR_NULL_PTR;
    if (tokens > kMaxCopies / top_k) return GG_ERR_BAD_SHAPE;
    if ((in_dtype != GG_DT_F32 && in_dtype != GG_DT_BF16) || (out_dtype != GG_DT_F32 && out_dtype != GG_DT_BF16))
        return GG_ERR_BAD_DTYPE;
    if (tokens * n > 0 && (!y || !out)) return GG_ERR_NULL_PTR;
    if (!aligned(y, elem_bytes(in_dtype)) || !aligned(out, elem_bytes(out_dtype)) || !aligned(copy_to_sorted, 4) ||
        !aligned(weights, 4))
        return GG_ERR_MISALIGNED;
    return launched(gg::launch_combine(y, in_dtype == GG_DT_BF16, (int)(tokens * top_k), copy_to_sorted, weights, (int)tokens,
                              top_k, (int)n, out, out_dtype == GG_DT_BF16, (hipStream_t)stream));
}

gg_status moe_permute_grad(const void* dsorted, const int32_t* copy_to_sorted, void* dx, int64_t tokens, int32_t top_k,
                           int64_t k, gg_dtype in_dtype, gg_dtype out_dtype, void* stream) {
    if (tokens < 0 || top_k < 1 || k < 0 || !fits_i32(k)) return GG_ERR_BAD_SHAPE;
    if (tokens > kMaxCopies / top_k) return GG_ERR_BAD_SHAPE;
    if ((in_dtype != GG_DT_F32 && in_dtype != GG_DT_BF16) || (out_dtype != GG_DT_F32 && out_dtype != GG_DT_BF16))
        return GG_ERR_BAD_DTYPE;
    if (tokens * k > 0 && (!copy_to_sorted || !dsorted || !dx)) return GG_ERR_NULL_PTR;
    if (!aligned(dsorted, elem_bytes(in_dtype)) || !aligned(dx, elem_bytes(out_dtype)) || !aligned(copy_to_sorted, 4))
        return GG_ERR_MISALIGNED;
    const uint64_t copies = (uint64_t)tokens * top_k, dx_bytes = (uint64_t)tokens * k * elem_bytes(out_dtype);
    if (overlap(dx, dx_bytes, dsorted, copies * k * elem_bytes(in_dtype)) || overlap(dx, dx_bytes, copy_to_sorted, copies * 4))
        return GG_ERR_UNSUPPORTED;
    return launched(gg::launch_combine(dsorted, in_dtype == GG_DT_BF16, (int)(tokens * top_k), copy_to_sorted, nullptr, (int)tokens,
                              top_k, (int)k, dx, out_dtype == GG_DT_BF16, (hipStream_t)stream));
}

gg_status moe_unpermute_grad(const void* dout, const void* y, const int32_t* copy_to_sorted, const int32_t* sorted_to_copy,
                             const float* weights, void* dy, float* dweights, int64_t tokens, int32_t top_k, int64_t n,
                             gg_dtype dtype, void* stream) {
    if (tokens < 0 || top_k < 1 || n < 0 || !fits_i32(n)) return GG_ERR_BAD_SHAPE;
    if (tokens > kMaxCopies / top_k) return GG_ERR_BAD_SHAPE;
    if (dtype != GG_DT_F32 && dtype != GG_DT_BF16) return GG_ERR_BAD_DTYPE;
    if (tokens > 0 && (!copy_to_sorted || !sorted_to_copy || !weights || !dweights)) return GG_ERR_NULL_PTR;
    if (tokens * n > 0 && (!dout || !y || !dy)) return GG_ERR_NULL_PTR;
    const size_t es = elem_bytes(dtype);
    if (!aligned(dout, es) || !aligned(y, es) || !aligned(dy, es) || !aligned(copy_to_sorted, 4) ||
        !aligned(sorted_to_copy, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return GG_ERR_MISALIGNED;
    const uint64_t copies = (uint64_t)tokens * top_k, dout_bytes = (uint64_t)tokens * n * es, rows_bytes = copies * n * es;
    auto on_inputs = [&](const void* p, uint64_t bytes) {
        return overlap(p, bytes, dout, dout_bytes) || overlap(p, bytes, y, rows_bytes) ||
               overlap(p, bytes, copy_to_sorted, copies * 4) || overlap(p, bytes, sorted_to_copy, copies * 4);
    };
    if (on_inputs(dy, rows_bytes) || overlap(dy, rows_bytes, weights, copies * 4) || overlap(dy, rows_bytes, dweights, copies * 4) ||
        on_inputs(dweights, copies * 4) || (dweights != weights && overlap(dweights, copies * 4, weights, copies * 4)))
        return GG_ERR_UNSUPPORTED;
    gg::UnpermuteGradArgs a{};
    a.dout = dout; a.y = y; a.copy_to_sorted = copy_to_sorted; a.sorted_to_copy = sorted_to_copy; a.weights = weights;
    a.dy = dy; a.dweights = dweights; a.tokens = (int)tokens; a.top_k = top_k; a.n = (int)n;
    return launched(gg::launch_unpermute_grad(a, dtype == GG_DT_BF16, (hipStream_t)stream));
}

gg_status mxfp4_quantize(const void* x, uint8_t* codes, uint8_t* scale, int64_t rows, int64_t k, int64_t x_stride,
                         gg_dtype in_dtype, void* stream) {
    // rows * panels bounds the launch and keeps every index of the kernels inside 63 bits
    if (rows < 0 || k < 0 || !fits_i32(rows) || !fits_i32(k) || x_stride < k || x_stride > (int64_t(1) << 31) ||
        !fits_i32(rows * cdiv64(k, 256)))
        return GG_ERR_BAD_SHAPE;
    if (in_dtype != GG_DT_F32 && in_dtype != GG_DT_BF16) return GG_ERR_BAD_DTYPE;
    if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if (rows * k > 0 && (!x || !codes || !scale)) return GG_ERR_NULL_PTR;
    if (!aligned(x, elem_bytes(in_dtype)) || !aligned(codes, 16) || !aligned(scale, 8)) return GG_ERR_MISALIGNED;
    return launched(gg::launch_fp4_quantize(x, in_dtype == GG_DT_BF16, rows, k, x_stride, codes, scale, (hipStream_t)stream));
}

gg_status mxfp4_quantize_weights(const void* w, uint8_t* codes, uint8_t* scale, int32_t g, int64_t k, int64_t n,
                                 gg_dtype in_dtype, void* stream) {
    if (k < 0 || n < 0 || g < 1 || g > GG_MAX_GROUPS || !fits_i32(k) || !fits_i32(n) || !fits_i32(n * cdiv64(k, 256)) ||
        !fits_i32(n * cdiv64(k, 256) * g))
        return GG_ERR_BAD_SHAPE;
    if (in_dtype != GG_DT_F32 && in_dtype != GG_DT_BF16) return GG_ERR_BAD_DTYPE;
    if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if (k * n > 0 && (!w || !codes || !scale)) return GG_ERR_NULL_PTR;
    if (!aligned(w, elem_bytes(in_dtype)) || !aligned(codes, 16) || !aligned(scale, 8)) return GG_ERR_MISALIGNED;
    return launched(gg::launch_fp4_quantize_weights(w, in_dtype == GG_DT_BF16, g, k, n, codes, scale, (hipStream_t)stream));
}

gg_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scale, void* out, int32_t g, int64_t n, int64_t k,
                           gg_dtype out_dtype, void* stream) {
    if (k < 0 || n < 0 || g < 1 || g > GG_MAX_GROUPS || !fits_i32(k) || !fits_i32(n) || !fits_i32(n * cdiv64(k, 256)) ||
        !fits_i32(n * cdiv64(k, 256) * g))
        return GG_ERR_BAD_SHAPE;
    if (out_dtype != GG_DT_F32 && out_dtype != GG_DT_BF16) return GG_ERR_BAD_DTYPE;
    if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if (k * n > 0 && (!codes || !scale || !out)) return GG_ERR_NULL_PTR;
    if (!aligned(out, elem_bytes(out_dtype)) || !aligned(codes, 16) || !aligned(scale, 8)) return GG_ERR_MISALIGNED;
    return launched(gg::launch_fp4_dequantize(codes, scale, g, n, k, out, out_dtype == GG_DT_BF16, (hipStream_t)stream));
}

gg_status ragged_dot_m_mxfp4(const void* lhs, const void* rhs, const int32_t* group_sizes, void* out, int64_t m, int64_t k,
                             int64_t n, int32_t g, gg_dtype out_dtype, const uint8_t* lhs_scale, const uint8_t* rhs_scale,
                             void* workspace, size_t workspace_bytes, void* stream) {
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes, kHeader);
    if (st != GG_OK) return st;
    if (out_dtype != GG_DT_BF16 && out_dtype != GG_DT_F32) return GG_ERR_BAD_DTYPE;
    if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if ((m * k > 0 && (!lhs || !lhs_scale)) || (k * n > 0 && (!rhs || !rhs_scale)) || (m * n > 0 && !out)) return GG_ERR_NULL_PTR;
    if (!aligned(lhs, 16) || !aligned(rhs, 16) || !aligned(lhs_scale, 8) || !aligned(rhs_scale, 8) ||
        !aligned(out, elem_bytes(out_dtype)))
        return GG_ERR_MISALIGNED;
    gg::Fp4Params p{};
    p.lhs = (const uint8_t*)lhs; p.rhs = (const uint8_t*)rhs; p.lhs_scale = lhs_scale; p.rhs_scale = rhs_scale;
    p.group_sizes = group_sizes; p.out = out; p.status = (uint32_t*)workspace;
    p.m = (int)m; p.k = (int)k; p.n = (int)n; p.g = g; p.out_f32 = out_dtype == GG_DT_F32;
    if (!gg::ragged_m_fp4_grid_ok(p)) return GG_ERR_BAD_SHAPE;
    int cus;
    if (device_cus(&cus) != 0) return GG_ERR_HIP;
    return gg::launch_ragged_m_fp4(p, cus, (hipStream_t)stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

int32_t gg_mxfp4_kernel(int64_t m, int64_t k, int64_t n, int32_t g, int32_t cus) {
    if (g < 1 || g > GG_MAX_GROUPS || cus < 1 || !fits_i32(m) || !fits_i32(k) || !fits_i32(n) || k % 32 != 0) return -1;
    gg::Fp4Params p{};
    p.m = (int)m; p.k = (int)k; p.n = (int)n; p.g = g;
    return gg::ragged_m_fp4_grid_ok(p) ? (int32_t)gg::ragged_m_fp4_kernel(p, cus) : -1;
}

gg_status mxfp8_quantize(const void* x, uint8_t* codes, uint8_t* scale, int64_t rows, int64_t k, int64_t x_stride,
                         gg_dtype in_dtype, void* stream) {
    if (!eights_ok(rows, k) || x_stride < k || x_stride > (int64_t(1) << 31)) return GG_ERR_BAD_SHAPE;
    if (!floats(in_dtype)) return GG_ERR_BAD_DTYPE;
    if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if (rows * k > 0 && (!x || !codes || !scale)) return GG_ERR_NULL_PTR;
    const size_t es = elem_bytes(in_dtype);
    if (!aligned(x, es) || !aligned(codes, 16)) return GG_ERR_MISALIGNED;
    const Span xs{x, (uint64_t)rows, (uint64_t)k * es, (uint64_t)x_stride * es}, cs = dense(codes, (uint64_t)(rows * k)),
               ss = dense(scale, (uint64_t)(rows * (k / 32)));
    if (meets(cs, xs, ss) || meets(ss, xs)) return GG_ERR_UNSUPPORTED;
    return launched(gg::launch_fp8_quantize(x, in_dtype == GG_DT_BF16, rows, k, x_stride, codes, scale, (hipStream_t)stream));
}

gg_status mxfp8_dequantize(const uint8_t* codes, const uint8_t* scale, void* out, int64_t rows, int64_t k, gg_dtype out_dtype,
                           void* stream) {
    if (!eights_ok(rows, k)) return GG_ERR_BAD_SHAPE;
    if (!floats(out_dtype)) return GG_ERR_BAD_DTYPE;
    if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if (rows * k > 0 && (!codes || !scale || !out)) return GG_ERR_NULL_PTR;
    const size_t es = elem_bytes(out_dtype);
    if (!aligned(codes, 16) || !aligned(out, es)) return GG_ERR_MISALIGNED;
    if (meets(dense(out, (uint64_t)(rows * k) * es), dense(codes, (uint64_t)(rows * k)), dense(scale, (uint64_t)(rows * (k / 32)))))
        return GG_ERR_UNSUPPORTED;
    return launched(gg::launch_fp8_dequantize(codes, scale, rows, k, out, out_dtype == GG_DT_BF16, (hipStream_t)stream));
}

gg_status gated_act_mxfp8(const void* gate, const void* up, void* h, uint8_t* codes, uint8_t* scale, int64_t m, int64_t n,
                          int64_t stride, gg_activation act, gg_dtype in_dtype, gg_dtype out_dtype, void* stream) {
    if (!eights_ok(m, n) || !eights_ok(m, 2 * n) || stride < n || stride > (int64_t(1) << 31)) return GG_ERR_BAD_SHAPE;
    if (!floats(in_dtype) || !floats(out_dtype)) return GG_ERR_BAD_DTYPE;
    if (n % 32 != 0 || (act != GG_ACT_SILU && act != GG_ACT_GELU_TANH)) return GG_ERR_UNSUPPORTED;
    if (m * n > 0 && (!gate || !up || !h || !codes || !scale)) return GG_ERR_NULL_PTR;
    const uint64_t es = elem_bytes(in_dtype), os = elem_bytes(out_dtype), M = (uint64_t)m, N = (uint64_t)n;
    if (!aligned(gate, es) || !aligned(up, es) || !aligned(h, os) || !aligned(codes, 16)) return GG_ERR_MISALIGNED;
    const Span g{gate, M, N * es, (uint64_t)stride * es}, u{up, M, N * es, (uint64_t)stride * es};
    const Span hs = dense(h, M * N * os), cs = dense(codes, 2 * M * N), ss = dense(scale, M * N / 16);
    if (meets(hs, g, u, cs, ss) || meets(cs, g, u, ss) || meets(ss, g, u)) return GG_ERR_UNSUPPORTED;
    gg::GatedActArgs a{};
    a.gate = gate; a.up = up; a.h = h; a.codes = codes; a.scale = scale; a.m = m; a.n = n; a.stride = stride;
    a.bf16 = in_dtype == GG_DT_BF16; a.out_bf16 = out_dtype == GG_DT_BF16; a.gelu = act == GG_ACT_GELU_TANH;
    return launched(gg::launch_gated_act(a, (hipStream_t)stream));
}

gg_status gated_act_mxfp8_grad(const void* dh, const uint8_t* codes, const uint8_t* scale, void* dgate, void* dup, void* h,
                               int64_t m, int64_t n, int64_t stride, gg_activation act, gg_dtype in_dtype, gg_dtype out_dtype,
                               void* stream) {
    if (!eights_ok(m, n) || !eights_ok(m, 2 * n) || stride < n || stride > (int64_t(1) << 31)) return GG_ERR_BAD_SHAPE;
    if (!floats(in_dtype) || !floats(out_dtype)) return GG_ERR_BAD_DTYPE;
    if (n % 32 != 0 || (act != GG_ACT_SILU && act != GG_ACT_GELU_TANH)) return GG_ERR_UNSUPPORTED;
    if (m * n > 0 && (!dh || !dgate || !dup || !codes || !scale)) return GG_ERR_NULL_PTR;
    const uint64_t es = elem_bytes(in_dtype), os = elem_bytes(out_dtype), M = (uint64_t)m, N = (uint64_t)n;
    if (!aligned(dh, es) || !aligned(dgate, os) || !aligned(dup, os) || !aligned(h, os) || !aligned(codes, 16)) return GG_ERR_MISALIGNED;
    const Span ds = dense(dh, M * N * es), cs = dense(codes, 2 * M * N), ss = dense(scale, M * N / 16);
    const Span g{dgate, M, N * os, (uint64_t)stride * os}, u{dup, M, N * os, (uint64_t)stride * os}, hs = dense(h, M * N * os);
    if (meets(g, cs, ss, u, hs) || meets(u, cs, ss, hs) || meets(hs, cs, ss)) return GG_ERR_UNSUPPORTED;
    // an element of dh is read by the lane that writes its place
    const bool same = in_dtype == out_dtype;
    if ((overlap(g, ds) && !(same && dgate == dh && stride == n)) || (overlap(u, ds) && !(same && dup == dh && stride == n)) ||
        (overlap(hs, ds) && !(same && h == dh)))
        return GG_ERR_UNSUPPORTED;
    gg::GatedActGradArgs a{};
    a.dh = dh; a.codes = codes; a.scale = scale; a.dgate = dgate; a.dup = dup; a.h = h; a.m = m; a.n = n; a.stride = stride;
    a.bf16 = in_dtype == GG_DT_BF16; a.out_bf16 = out_dtype == GG_DT_BF16; a.gelu = act == GG_ACT_GELU_TANH;
    return launched(gg::launch_gated_act_grad(a, (hipStream_t)stream));
}

gg_status ragged_dot_k_mxfp8(const void* lhs, const uint8_t* lhs_scale, const void* dout, const int32_t* group_sizes, void* out,
                             int64_t m, int64_t k, int64_t n, int32_t g, gg_dtype out_dtype, float alpha, float beta,
                             void* workspace, size_t workspace_bytes, void* stream) {
    gg_status st = check_common(m, k, n, g, group_sizes, workspace, workspace_bytes,
                                gg_workspace_bytes(GG_OP_RAGGED_K, m, k, n, g, 0, GG_DT_E4M3));
    if (st != GG_OK) return st;
    if (!floats(out_dtype)) return GG_ERR_BAD_DTYPE;
    if (k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if ((m * k > 0 && (!lhs || !lhs_scale)) || (m * n > 0 && !dout) || (k * n > 0 && !out)) return GG_ERR_NULL_PTR;
    if (!aligned(lhs, 16) || !aligned(dout, 2) || !aligned(out, elem_bytes(out_dtype))) return GG_ERR_MISALIGNED;
    int cus;
    if (device_cus(&cus) != 0) return GG_ERR_HIP;
    const int splits = gg::ragged_k_mx_splits(m, k, n, g);
    const int64_t bound = (int64_t)g * splits * cdiv64(k, 128) * cdiv64(n, 256);   // tiles of the smallest size
    if (!fits_i32(bound)) return GG_ERR_BAD_SHAPE;
    gg::KmxParams p{};
    p.lhs = (const uint8_t*)lhs; p.lhs_scale = lhs_scale; p.dout = (const uint16_t*)dout; p.group_sizes = group_sizes; p.out = out;
    p.status = (uint32_t*)workspace; p.m = (int)m; p.k = (int)k; p.n = (int)n; p.g = g; p.out_f32 = out_dtype == GG_DT_F32;
    p.alpha = alpha; p.beta = beta; p.splits = splits; p.parts = (float*)((char*)workspace + kHeader);
    return gg::launch_ragged_k_mx(p, cus, (hipStream_t)stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

gg_status ragged_lora(const void* x, const void* a, const void* b, const int32_t* group_sizes, const int32_t* row_group,
                      const float* scaling, const void* base, void* out, float* v, int64_t m, int64_t k, int64_t n, int32_t r,
                      int32_t g, int64_t x_stride, int64_t base_stride, int64_t out_stride, gg_dtype dtype, gg_dtype out_dtype,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (!group_sizes == !row_group && m > 0) return group_sizes ? GG_ERR_UNSUPPORTED : GG_ERR_NULL_PTR;
    if (!workspace) return GG_ERR_NULL_PTR;
    if (m < 0 || k < 0 || n < 0 || g < 1 || g > GG_MAX_GROUPS || !fits_i32(m) || !fits_i32(k) || !fits_i32(n) || r < 1 ||
        r > GG_MAX_RANK || x_stride < k || (base && base_stride < n) || out_stride < n || x_stride > (int64_t(1) << 31) ||
        base_stride > (int64_t(1) << 31) || out_stride > (int64_t(1) << 31))
        return GG_ERR_BAD_SHAPE;
    if (!floats(dtype) || !floats(out_dtype)) return GG_ERR_BAD_DTYPE;
    if ((m * k > 0 && !x) || (m > 0 && k > 0 && !a) || (m > 0 && n > 0 && (!b || !out))) return GG_ERR_NULL_PTR;
    const uint64_t es = elem_bytes(dtype), os = elem_bytes(out_dtype), M = (uint64_t)m;
    if (!aligned(x, es) || !aligned(a, es) || !aligned(b, es) || !aligned(group_sizes, 4) || !aligned(row_group, 4) ||
        !aligned(scaling, 4) || !aligned(base, os) || !aligned(out, os) || !aligned(v, 4) || !aligned(workspace, 16))
        return GG_ERR_MISALIGNED;
    const size_t need = gg_workspace_bytes(GG_OP_LORA, m, k, n, g, r, dtype);
    if (workspace_bytes < need) return GG_ERR_WORKSPACE_TOO_SMALL;
    if (m == 0) return GG_OK;
    const Span xs{x, M, (uint64_t)k * es, (uint64_t)x_stride * es}, as = dense(a, (uint64_t)g * r * k * es),
               bs = dense(b, (uint64_t)g * n * r * es), ids = group_sizes ? dense(group_sizes, 4ull * g) : dense(row_group, 4 * M),
               sc = dense(scaling, 4ull * g), bas{base, M, (uint64_t)n * os, (uint64_t)base_stride * os},
               outs{out, M, (uint64_t)n * os, (uint64_t)out_stride * os}, vs = dense(v, 4 * M * r), wss = dense(workspace, need);
    const bool in_place = base == out && base_stride == out_stride;
    if (meets(outs, xs, as, bs, ids, sc, vs, wss) || (!in_place && meets(outs, bas)) || meets(vs, xs, as, bs, ids, sc, bas, wss) ||
        meets(wss, xs, as, bs, ids, sc, bas))
        return GG_ERR_UNSUPPORTED;
    gg::lora::Rows rows{};
    rows.group_sizes = group_sizes; rows.row_group = row_group; rows.status = (uint32_t*)workspace; rows.m = (int)m; rows.g = g;
    gg::lora_rows(rows);
    if (!gg::lora_grid_ok(rows, n)) return GG_ERR_BAD_SHAPE;
    const int splits = gg::lora_splits(m, k, r, g);
    float* t = splits == 1 && v ? v : (float*)((char*)workspace + kHeader);
    gg::lora::Shrink sh{rows, x, a, t, x_stride, (int)k, r, splits};
    if (gg::lora_both_ok(sh, dtype == GG_DT_BF16)) {
        const gg::lora::Expand ex{rows, nullptr, b, scaling, base, out, v, base_stride, out_stride, (int)n, r, 0, 0, 0};
        return launched(gg::launch_lora_both(sh, ex, dtype == GG_DT_BF16, out_dtype == GG_DT_BF16, (hipStream_t)stream));
    }
    hipError_t e = gg::launch_lora_shrink(sh, dtype == GG_DT_BF16, (hipStream_t)stream);
    if (e != hipSuccess) return launched(e);
    rows.status = nullptr;
    gg::lora::Expand ex{rows, t, b, scaling, base, out, v, base_stride, out_stride, (int)n, r, splits, 0, 0};
    return launched(gg::launch_lora_expand(ex, dtype == GG_DT_BF16, out_dtype == GG_DT_BF16, (hipStream_t)stream));
}

gg_status ragged_lora_grad(const void* x, const uint8_t* x_scale, const float* v, const void* dout, const void* a, const void* b,
                           const int32_t* group_sizes, const float* scaling, const void* dbase, void* dx, void* da, void* db,
                           int64_t m, int64_t k, int64_t n, int32_t r, int32_t g, gg_dtype x_dtype, gg_dtype dtype,
                           gg_dtype grad_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!group_sizes || !workspace) return GG_ERR_NULL_PTR;
    gg_status st = check_shape(m, k, n, g, group_sizes);
    if (st != GG_OK) return st;
    if (r < 1 || r > GG_MAX_RANK) return GG_ERR_BAD_SHAPE;
    const bool e4m3 = x_dtype == GG_DT_E4M3;
    if (!floats(dtype) || !floats(grad_dtype) || (e4m3 ? dtype != GG_DT_BF16 : x_dtype != dtype)) return GG_ERR_BAD_DTYPE;
    if (!e4m3 && x_scale) return GG_ERR_BAD_DTYPE;
    if (e4m3 && k % 32 != 0) return GG_ERR_UNSUPPORTED;
    if ((m * k > 0 && (!x || (e4m3 && !x_scale))) || (m > 0 && !v) || (m * n > 0 && !dout) || (k > 0 && (!a || !da)) ||
        (n > 0 && (!b || !db)) || (dbase && !dx))
        return GG_ERR_NULL_PTR;
    const uint64_t es = elem_bytes(dtype), gs = elem_bytes(grad_dtype), xb = elem_bytes(x_dtype), M = (uint64_t)m, K = (uint64_t)k,
                   N = (uint64_t)n, G = (uint64_t)g * r;
    if (!aligned(x, e4m3 ? 16 : es) || !aligned(v, 4) || !aligned(dout, es) || !aligned(a, es) || !aligned(b, es) ||
        !aligned(scaling, 4) || !aligned(dbase, es) || !aligned(dx, es) || !aligned(da, gs) || !aligned(db, gs) || !aligned(workspace, 16))
        return GG_ERR_MISALIGNED;
    const size_t need = gg_workspace_bytes(GG_OP_LORA_GRAD, m, k, n, g, r, dtype);
    if (need == 0) return GG_ERR_BAD_SHAPE;
    if (workspace_bytes < need) return GG_ERR_WORKSPACE_TOO_SMALL;
    const Span xs = dense(x, M * K * xb), xss = dense(x_scale, M * K / 32), vs = dense(v, 4 * M * r), dos = dense(dout, M * N * es),
               as = dense(a, G * K * es), bs = dense(b, G * N * es), ids = dense(group_sizes, 4ull * g), sc = dense(scaling, 4ull * g),
               dbs = dense(dbase, M * K * es), dxs = dense(dx, M * K * es), das = dense(da, G * K * gs), dbw = dense(db, G * N * gs),
               wss = dense(workspace, need);
    auto inputs = [&](const Span& o) { return meets(o, xs, xss, vs, dos, as, bs, ids, sc); };
    if (inputs(dxs) || inputs(das) || inputs(dbw) || inputs(wss) || (dbase != dx && meets(dxs, dbs)) || meets(das, dbs, dxs, dbw, wss) ||
        meets(dbw, dbs, dxs, wss) || meets(wss, dbs, dxs))
        return GG_ERR_UNSUPPORTED;
    const bool bf16 = dtype == GG_DT_BF16;
    hipStream_t s = (hipStream_t)stream;
    char* ws = (char*)workspace + kHeader;
    const LoraGradLayout w = lora_grad_layout(m, k, n, r, g, dtype);
    const int splits = gg::lora_splits(m, n, r, g);
    float* t = (float*)(ws + w.t);
    float* u = (float*)(ws + w.u);
    gg::lora::Rows rows{};
    rows.group_sizes = group_sizes; rows.m = (int)m; rows.g = g;
    gg::lora_rows(rows);
    if (!gg::lora_grid_ok(rows, k)) return GG_ERR_BAD_SHAPE;
    hipError_t e = gg::launch_lora_turn(b, ws + w.bt, (int)n, r, dx ? a : nullptr, ws + w.at, r, (int)k, bf16, g, s);
    if (e != hipSuccess) return launched(e);
    gg::lora::Shrink sh{rows, dout, ws + w.bt, t, n, (int)n, r, splits};
    const bool both = gg::lora_both_ok(sh, bf16);
    if (!both) e = gg::launch_lora_shrink(sh, bf16, s);
    if (e != hipSuccess) return launched(e);
    gg::lora::Expand ex{rows, t, ws + w.at, scaling, dbase, dx, splits > 1 ? u : nullptr, k, k, dx ? (int)k : 0, r, splits, 0, 0};
    gg::lora::Outer o{};
    o.group_sizes = group_sizes; o.status = (uint32_t*)workspace; o.x = x; o.x_scale = e4m3 ? x_scale : nullptr; o.dout = dout;
    o.u = u; o.v = v; o.scaling = scaling; o.parts = (float*)(ws + w.parts); o.da = da; o.db = db;
    o.m = (int)m; o.k = (int)k; o.n = (int)n; o.r = r; o.g = g; o.chunk = gg::lora_chunk(m, k, n); o.grads_bf16 = grad_dtype == GG_DT_BF16;
    // with splits the expand sums them for the row sums, so it goes first (without dx it does only that)
    if (both) {
        ex.v = u;
        e = gg::launch_lora_both(sh, ex, bf16, bf16, s);
    } else if (splits > 1) {
        e = gg::launch_lora_expand(ex, bf16, bf16, s);
    }
    if (e == hipSuccess) e = gg::launch_lora_outer(o, bf16, s);
    if (e == hipSuccess && !both && splits == 1 && dx) e = gg::launch_lora_expand(ex, bf16, bf16, s);
    return launched(e);
}

gg_status gg_schedule(const int32_t* group_sizes, int64_t m, int64_t n, int32_t g, int32_t block_m, int32_t block_n,
                      int32_t* row_off, int32_t* tile_off, uint32_t* status, void* stream) {
    if (!group_sizes || !row_off || !tile_off || !status) return GG_ERR_NULL_PTR;
    if (m < 0 || n < 0 || g < 1 || g > GG_MAX_GROUPS || !fits_i32(m) || !fits_i32(n)) return GG_ERR_BAD_SHAPE;
    if (block_m < 1 || block_m > 4096 || block_n < 1 || block_n > 4096) return GG_ERR_BAD_SHAPE;
    if (!aligned(group_sizes, 4) || !aligned(row_off, 4) || !aligned(tile_off, 4) || !aligned(status, 4))
        return GG_ERR_MISALIGNED;
    hipError_t e = gg::launch_schedule(group_sizes, (int)m, (int)n, g, block_m, block_n, row_off, tile_off, status,
                                       (hipStream_t)stream);
    return e == hipSuccess ? GG_OK : GG_ERR_HIP;
}

gg_status gg_read_device_status(const void* workspace, uint32_t* flags, void* stream) {
    if (!workspace || !flags) return GG_ERR_NULL_PTR;
    hipStream_t s = (hipStream_t)stream;
    if (hipStreamSynchronize(s) != hipSuccess) return GG_ERR_HIP;
    if (hipMemcpy(flags, workspace, sizeof(uint32_t), hipMemcpyDeviceToHost) != hipSuccess) return GG_ERR_HIP;
    return GG_OK;
}

}  // extern "C"
