// mxfp4.hip -- rows and weights to MXFP4 and back: OCP e2m1 codes, two per byte along k, and one E8M0
// scale per 32 elements, kept in panels [ceil(k/256), rows, 8] (groupgemm.h, "MXFP4 tensors").
//
// One block of 32 values x: with E the biased fp32 exponent of max |x|, the scale byte is
// b = max(E - 2, 0) (2 = exponent of e2m1's largest value 6), the codes are x * 2^(127 - b) rounded to
// nearest even and saturated at 6.  A non-finite value makes E = 255 and the byte 255, E8M0's NaN.
// gfx950 converts two values an instruction, scaled by the exponent field of an fp32 register:
// v_cvt_scalef32_pk_fp4_* rounds to nearest even and saturates, and takes field 0 as 2^-127 and field 255
// as NaN in both directions (checked on the GPU for every code at scale bytes 0-3, 100, 127, 128, 200 and
// 252-255), so one conversion is exact to the definition and the scale is one shift.
//
// All three kernels move each byte once and compute little: they are bound by memory.  Measured: rows
// [4096, 7168] bf16 12.8 us and back 12.0 us (5.8 and 6.2 TB/s, part of it out of the last-level cache), fp32 24.5
// and 23.4; weights [8, 4096, 14336] bf16 198 us and back 232 us (6.0 and 5.1 TB/s), fp32 359 and 598 us (5.9 and
// 3.6 TB/s: the way back to fp32 is 1.3 times a copy's time).
#include "common.hpp"
#include "launch.hpp"

namespace gg {
namespace fp4 {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kPanel = 256;   // elements along k whose 8 scale bytes lie together

// biased exponent of the largest magnitude -> scale byte
__device__ inline int scale_byte(uint32_t exponent) {
    const int e = (int)exponent;
    return e == 255 ? 255 : (e > 2 ? e - 2 : 0);
}

// eight values to one dword of codes (scale: an fp32 with the scale byte as its exponent field)
__device__ inline uint32_t encode8(const uint32_t (&v)[4], float scale) {   // bf16 pairs
    int q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, v[0]), scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, v[1]), scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, v[2]), scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, v[3]), scale, 3);
    return (uint32_t)q;
}
__device__ inline uint32_t encode8(const float (&v)[8], float scale) {
    int q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
    return (uint32_t)q;
}

// 16 bytes of a row, which may begin at any element (the target's global memory takes that)
typedef i32x4 __attribute__((aligned(2))) i32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

// Eight consecutive values of a row, and the exponent of their largest magnitude.
template <typename T> struct Eight;
template <> struct Eight<uint16_t> {
    uint32_t v[4];
    __device__ void load(const uint16_t* p) {
        const i32x4 q = *(const i32x4_any*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (uint32_t)q[i];
    }
    __device__ void zero() { v[0] = v[1] = v[2] = v[3] = 0; }
    __device__ uint32_t top() const {   // magnitudes order as integers, NaN above infinity
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
        return m >> 7;
    }
};
template <> struct Eight<float> {
    float v[8];
    __device__ void load(const float* p) {
        const f32x4 a = *(const f32x4_any*)p, b = *(const f32x4_any*)(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    }
    __device__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    __device__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        return m >> 23;
    }
};

// Rows.  A half wave holds one panel of one row, eight elements a lane, so a block is four lanes and its
// maximum two lane exchanges.  A workgroup takes 8 U rows of one panel, so the panel's scale bytes of its
// rows leave as one contiguous run and U loads a lane are in flight.
template <typename T, int U>
__global__ __launch_bounds__(256) void quantize_rows(const T* __restrict__ x, int64_t rows, int64_t k, int64_t stride,
                                                     uint8_t* __restrict__ codes, uint8_t* __restrict__ scale, int panels) {
    const int t = threadIdx.x, c = t & 31, sub = t >> 5;
    const int p = blockIdx.x % panels;
    const int64_t r0 = (int64_t)(blockIdx.x / panels) * (8 * U) + sub;
    const int64_t col = (int64_t)p * kPanel + 8 * c;
    Eight<T> e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + 8 * u;
        if (r < rows && col < k) e[u].load(x + r * stride + col);
        else e[u].zero();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + 8 * u;
        uint32_t m = e[u].top();
        m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
        const int b = scale_byte(m);
        const uint32_t q = encode8(e[u].v, __uint_as_float((uint32_t)b << 23));
        // the panel's eight bytes, gathered from lanes 0, 4, .., 28 of the half wave
        uint32_t w = (uint32_t)b << (8 * ((c >> 2) & 3));
        w |= (uint32_t)__shfl_xor((int)w, 4, 64);
        w |= (uint32_t)__shfl_xor((int)w, 8, 64);
        if (r < rows) {
            if (col < k) *(uint32_t*)(codes + r * (k >> 1) + (col >> 1)) = q;
            if ((c & 15) == 0) *(uint32_t*)(scale + ((int64_t)p * rows + r) * 8 + (c >> 2)) = w;
        }
    }
}

// Weights [g, k, n] -> codes [g, n, k/2].  A thread holds 16 bytes of columns (8 bf16 or 4 fp32) of the 32
// rows of one block, so a column's maximum and its 32 codes need no exchange; a workgroup holds one panel
// (8 blocks) of 32 threads' columns.  The codes turn in LDS and leave as the panel's 128 bytes of every
// column, whole cache lines.
template <typename T>
__global__ __launch_bounds__(256) void quantize_weights(const T* __restrict__ w, int64_t k, int64_t n, int panels, int ntiles,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scale) {
    constexpr int C = 16 / sizeof(T), COLS = 32 * C;
    __shared__ i32x4 turn[COLS * 8];
    __shared__ __attribute__((aligned(8))) uint8_t sbytes[COLS * 8];
    const int t = threadIdx.x, cg = t & 31, blk = t >> 5;
    const int nt = blockIdx.x % ntiles;
    const int p = (blockIdx.x / ntiles) % panels;
    const int64_t h = blockIdx.x / ntiles / panels;
    // (a row's last 16 bytes may begin before their place: the columns that two threads hold come out the same)
    const int64_t col0 = (int64_t)nt * COLS, col = n < C ? C * cg : min(col0 + C * cg, n - C);
    const int64_t k0 = (int64_t)p * kPanel + 32 * blk;
    const T* src = w + (h * k + k0) * n + col;
    uint32_t v[32][4];   // row i of the block: the thread's C columns
    if (k0 < k && n >= C) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const i32x4 q = __builtin_nontemporal_load((const i32x4_any*)(src + (int64_t)i * n));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = (uint32_t)q[j];
        }
    } else {   // fewer columns than that, and blocks past k
#pragma unroll
        for (int i = 0; i < 32; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = 0;
            if (k0 >= k) continue;
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (col + j < n) {
                    const T a = src[(int64_t)i * n + j];
                    if constexpr (sizeof(T) == 2) v[i][j >> 1] |= (uint32_t)a << (16 * (j & 1));
                    else v[i][j] = __float_as_uint((float)a);
                }
        }
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
        uint32_t m = 0;
        i32x4 q;
        int b;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 32; ++i) m = max(m, (v[i][j >> 1] >> (16 * (j & 1))) & 0x7fffu);
            b = scale_byte(m >> 7);
            const float s = __uint_as_float((uint32_t)b << 23);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                uint32_t pair[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // rows 8 d + 2 i and + 1 of column j
                    const uint32_t lo = v[8 * d + 2 * i][j >> 1], hi = v[8 * d + 2 * i + 1][j >> 1];
                    pair[i] = __builtin_amdgcn_perm(hi, lo, (j & 1) ? 0x07060302u : 0x05040100u);
                }
                q[d] = (int)encode8(pair, s);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) m = max(m, v[i][j] & 0x7fffffffu);
            b = scale_byte(m >> 23);
            const float s = __uint_as_float((uint32_t)b << 23);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[8 * d + i][j]);
                q[d] = (int)encode8(x, s);
            }
        }
        const int cl = (int)(col - col0) + j;
        if (cl < 0) continue;
        turn[cl * 8 + (blk ^ ((cl / C) & 7))] = q;   // 16-byte chunk of the column, spread over the banks
        sbytes[cl * 8 + blk] = (uint8_t)(k0 < k ? b : 0);
    }
    __syncthreads();
    const int chunk = t & 7;
#pragma unroll
    for (int u = 0; u < COLS / 32; ++u) {
        const int cl = 32 * u + (t >> 3);
        const int64_t byte = (int64_t)p * (kPanel / 2) + 16 * chunk;
        if (col0 + cl < n && byte < (k >> 1))
            *(i32x4*)(codes + (h * n + col0 + cl) * (k >> 1) + byte) = turn[cl * 8 + (chunk ^ ((cl / C) & 7))];
    }
    if (t < COLS && col0 + t < n)
        *(i32x2*)(scale + ((h * panels + p) * n + col0 + t) * 8) = *(const i32x2*)(sbytes + 8 * t);
}

// Back to values, the geometry of quantize_rows: a lane turns one dword of codes into eight values.
template <typename OutT, int U>
__global__ __launch_bounds__(256) void dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scale, int64_t n,
                                                  int64_t k, int panels, int rtiles, OutT* __restrict__ out) {
    const int t = threadIdx.x, c = t & 31, sub = t >> 5;
    const int p = blockIdx.x % panels;
    const int64_t h = blockIdx.x / panels / rtiles;
    const int64_t r0 = (int64_t)((blockIdx.x / panels) % rtiles) * (8 * U) + sub;
    const int64_t col = (int64_t)p * kPanel + 8 * c;
    if (col >= k) return;
    uint32_t q[U];
    uint8_t b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + 8 * u;
        q[u] = 0;
        b[u] = 0;
        if (r < n) {
            q[u] = *(const uint32_t*)(codes + (h * n + r) * (k >> 1) + (col >> 1));
            b[u] = scale[((h * panels + p) * n + r) * 8 + (c >> 2)];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + 8 * u;
        if (r >= n) continue;
        const float s = __uint_as_float((uint32_t)b[u] << 23);
        OutT* o = out + (h * n + r) * k + col;
        if constexpr (sizeof(OutT) == 2) {
            i32x4 v;
            v[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s, 0));
            v[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s, 1));
            v[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s, 2));
            v[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s, 3));
            *(i32x4_any*)o = v;
        } else {
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 0), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 1);
            const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 3);
            *(f32x4_any*)o = f32x4{a[0], a[1], e[0], e[1]};
            *(f32x4_any*)(o + 4) = f32x4{f[0], f[1], d[0], d[1]};
        }
    }
}

template <typename T>
hipError_t quantize_t(const void* x, int64_t rows, int64_t k, int64_t stride, uint8_t* codes, uint8_t* scale, hipStream_t s) {
    const int panels = (int)((k + kPanel - 1) / kPanel);
    constexpr int U = 4;
    const int64_t grid = (rows + 8 * U - 1) / (8 * U) * panels;
    if (grid > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((quantize_rows<T, U>), dim3((uint32_t)grid), dim3(256), 0, s, (const T*)x, rows, k, stride, codes, scale, panels);
    return hipGetLastError();
}

template <typename T>
hipError_t quantize_weights_t(const void* w, int g, int64_t k, int64_t n, uint8_t* codes, uint8_t* scale, hipStream_t s) {
    const int panels = (int)((k + kPanel - 1) / kPanel);
    constexpr int COLS = 32 * 16 / sizeof(T);
    const int64_t ntiles = (n + COLS - 1) / COLS;
    const int64_t grid = ntiles * panels * g;
    if (grid > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((quantize_weights<T>), dim3((uint32_t)grid), dim3(256), 0, s, (const T*)w, k, n, panels, (int)ntiles, codes, scale);
    return hipGetLastError();
}

template <typename OutT>
hipError_t dequantize_t(const uint8_t* codes, const uint8_t* scale, int g, int64_t n, int64_t k, void* out, hipStream_t s) {
    const int panels = (int)((k + kPanel - 1) / kPanel);
    constexpr int U = 4;
    const int64_t rtiles = (n + 8 * U - 1) / (8 * U);
    const int64_t grid = rtiles * panels * g;
    if (grid > kMaxBlocks) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((dequantize<OutT, U>), dim3((uint32_t)grid), dim3(256), 0, s, codes, scale, n, k, panels, (int)rtiles, (OutT*)out);
    return hipGetLastError();
}

}  // namespace fp4

hipError_t launch_fp4_quantize(const void* x, bool bf16, int64_t rows, int64_t k, int64_t stride, uint8_t* codes,
                               uint8_t* scale, hipStream_t s) {
    if (rows == 0 || k == 0) return hipSuccess;
    return bf16 ? fp4::quantize_t<uint16_t>(x, rows, k, stride, codes, scale, s) : fp4::quantize_t<float>(x, rows, k, stride, codes, scale, s);
}

hipError_t launch_fp4_quantize_weights(const void* w, bool bf16, int g, int64_t k, int64_t n, uint8_t* codes, uint8_t* scale,
                                       hipStream_t s) {
    if (k == 0 || n == 0) return hipSuccess;
    return bf16 ? fp4::quantize_weights_t<uint16_t>(w, g, k, n, codes, scale, s) : fp4::quantize_weights_t<float>(w, g, k, n, codes, scale, s);
}

hipError_t launch_fp4_dequantize(const uint8_t* codes, const uint8_t* scale, int g, int64_t n, int64_t k, void* out,
                                 bool out_bf16, hipStream_t s) {
    if (k == 0 || n == 0) return hipSuccess;
    return out_bf16 ? fp4::dequantize_t<uint16_t>(codes, scale, g, n, k, out, s) : fp4::dequantize_t<float>(codes, scale, g, n, k, out, s);
}

}  // namespace gg
