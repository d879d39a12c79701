// mxfp8.hip -- activation checkpoints in 8 bits: rows to MXFP8 (OCP e4m3, one E8M0 scale per 32 elements)
// and back, and the gated unit of an expert block that keeps its two inputs that way.
//
// One block of 32 values x: with E the biased fp32 exponent of max |x| and F its fraction, the scale byte is
// b = max(E - 8 + (F > 0.75), 0), the smallest power of two with which no value passes e4m3's 448 = 1.75 * 2^8,
// and the codes are x * 2^(127 - b) rounded to nearest even, so nothing is clipped and a code's error is at
// most 2^-4 of its value (2^-10 of the scale's power where the code is subnormal).  A non-finite value makes
// the byte 255, E8M0's NaN: the whole block reads as NaN.
//
// The gated unit, with y = gate for SiLU and 2 sqrt(2/pi) (gate + 0.044715 gate^3) for tanh-GELU (0.5 (1 + tanh z)
// is the logistic function of 2 z), p = 1 / (1 + e^-y):
//   h = gate p up;   dgate = dh up (p + gate p (1 - p) y'),   dup = dh gate p.
//
// All kernels move each byte once and are bound by memory; eight elements a lane, so a block is four lanes and
// its maximum two lane exchanges.  Measured in bf16, 16384 rows of 5120 values: to 8 bits in 41 us (254 MB) and back in 36;
// 8192 rows of width 14336: the unit with its checkpoint 140 us (947 MB with h), its gradient with h 193 (1182 MB; a copy's
// rate would be 236, but part of what the caller just wrote is still in the last-level cache).
#include "common.hpp"
#include "launch.hpp"

namespace gg {
namespace fp8 {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// 16 bytes that may begin at any element (the target's global memory takes that)
typedef i32x4 __attribute__((aligned(2))) i32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

// q = x / d for 0 <= x < 2^31 by one multiplication (Granlund and Montgomery, "Division by Invariant Integers
// using Multiplication", with the divisor's reciprocal rounded up)
struct Divisor {
    uint32_t d, mul, shift;
};
static Divisor divisor(uint32_t d) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    return {d, (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1), l};
}
__device__ inline uint32_t div_by(uint32_t x, const Divisor& v) { return (uint32_t)(((uint64_t)__umulhi(x, v.mul) + x) >> v.shift); }

// eight consecutive values of a row as fp32, from fp32 or bf16
template <typename T> struct Eight;
template <> struct Eight<uint16_t> {
    i32x4 q;
    __device__ void load(const uint16_t* p) { q = __builtin_nontemporal_load((const i32x4_any*)p); }
    __device__ float get(int i) const { return __uint_as_float((i & 1) ? (uint32_t)q[i >> 1] & 0xffff0000u : (uint32_t)q[i >> 1] << 16); }
    // bits of the largest magnitude, as fp32
    __device__ uint32_t top() const {   // magnitudes order as integers, NaN above infinity
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max((uint32_t)q[i] & 0x7fffu, ((uint32_t)q[i] >> 16) & 0x7fffu));
        return m << 16;
    }
};
template <> struct Eight<float> {
    f32x4 a, b;
    __device__ void load(const float* p) {
        a = __builtin_nontemporal_load((const f32x4_any*)p);
        b = __builtin_nontemporal_load((const f32x4_any*)(p + 4));
    }
    __device__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
    __device__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(get(i)) & 0x7fffffffu);
        return m;
    }
};
__device__ inline void store8(uint16_t* p, const float (&v)[8]) {
    i32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 w = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
        q[i] = __builtin_bit_cast(int, w);
    }
    __builtin_nontemporal_store(q, (i32x4_any*)p);
}
__device__ inline void store8(float* p, const float (&v)[8]) {
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4_any*)p);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4_any*)(p + 4));
}

// scale byte of the block that this lane shares with the three next to it
template <typename T>
__device__ inline int block_byte(const Eight<T>& e) {
    uint32_t m = e.top();
    m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
    const int E = (int)(m >> 23);
    return E == 255 ? 255 : max(E - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
}
// Eight codes.  The conversion takes the scale from an fp32 register's exponent field.  Byte 0 is 2^-127: values
// and scale are both taken 2^64 higher there, since all of such a block's values are below 2^-118.
template <typename T>
__device__ inline i32x2 encode8(const Eight<T>& e, int byte) {
    const float s = __uint_as_float((uint32_t)(byte < 64 ? byte + 64 : byte) << 23), up = byte < 64 ? 0x1p64f : 1.0f;
    i32x2 r;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        i16x2 c = {0, 0};
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, e.get(4 * d) * up, e.get(4 * d + 1) * up, s, false);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, e.get(4 * d + 2) * up, e.get(4 * d + 3) * up, s, true);
        r[d] = __builtin_bit_cast(int, c);
    }
    return r;
}
// 2^(byte - 127); 255 is NaN
__device__ inline float scale_value(int byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : (uint32_t)byte << 23);
}
__device__ inline void decode8(i32x2 c, int byte, float (&v)[8]) {
    const float s = scale_value(byte);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(c[d], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c[d], true);
        v[4 * d] = lo[0] * s; v[4 * d + 1] = lo[1] * s; v[4 * d + 2] = hi[0] * s; v[4 * d + 3] = hi[1] * s;
    }
}

// Rows of `per` eights; a lane takes eights i, i + 256, ... of its workgroup's 256 U.  Dense rows are one long row.
template <typename T, bool DENSE, int U>
__global__ __launch_bounds__(256) void quantize(const T* __restrict__ x, uint32_t eights, Divisor per, int64_t stride,
                                                uint8_t* __restrict__ codes, uint8_t* __restrict__ scale) {
    const uint32_t i0 = blockIdx.x * (256u * U) + threadIdx.x;
    Eight<T> e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = min(i0 + 256u * u, eights - 1);
        const uint32_t r = DENSE ? 0 : div_by(i, per);
        e[u].load(DENSE ? x + (size_t)i * 8 : x + (int64_t)r * stride + (int64_t)(i - r * per.d) * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + 256u * u;
        const int b = block_byte(e[u]);
        const i32x2 c = encode8(e[u], b);
        if (i < eights) {
            *(i32x2*)(codes + (size_t)i * 8) = c;
            if ((i & 3) == 0) scale[i >> 2] = (uint8_t)b;
        }
    }
}

template <typename T, int U>
__global__ __launch_bounds__(256) void dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scale, uint32_t eights,
                                                  T* __restrict__ out) {
    const uint32_t i0 = blockIdx.x * (256u * U) + threadIdx.x;
    i32x2 c[U];
    int b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = min(i0 + 256u * u, eights - 1);
        c[u] = *(const i32x2*)(codes + (size_t)i * 8);
        b[u] = scale[i >> 2];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + 256u * u;
        float v[8];
        decode8(c[u], b[u], v);
        if (i < eights) store8(out + (size_t)i * 8, v);
    }
}

// act(x) = x p(x) and its derivative.  Past |x| = 30 p is 0 or 1 in fp32 for both, so y and y' are taken at x held
// to that range, and e^-y, held to 2^127, stays finite: no product of an infinity and a zero.
struct Gate { float f, d; };
template <bool GELU>
__device__ inline Gate gate_of(float x) {
    float y = x, dy = 1.f;
    if constexpr (GELU) {
        const float c = fminf(fmaxf(x, -30.f), 30.f), a = 1.5957691216057308f;   // 2 sqrt(2 / pi)
        y = a * (c + 0.044715f * c * c * c);
        dy = a * (1.f + 0.134145f * c * c);
    }
    const float e = expf(fminf(-y, 88.f));
    const float p = __builtin_amdgcn_rcpf(1.f + e);
    return {x * p, p + x * p * (e * p) * dy};
}

struct GatedArgs {
    const void* gate;
    const void* up;
    void* h;
    uint8_t* codes;
    uint8_t* scale;
    uint32_t eights;
    Divisor per;
    int64_t stride;
};
template <typename T, typename H, bool GELU, int U>
__global__ __launch_bounds__(256) void gated(GatedArgs p) {
    const uint32_t i0 = blockIdx.x * (256u * U) + threadIdx.x;
    Eight<T> g[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = min(i0 + 256u * u, p.eights - 1), r = div_by(i, p.per);
        const int64_t at = (int64_t)r * p.stride + (int64_t)(i - r * p.per.d) * 8;
        g[u].load((const T*)p.gate + at);
        w[u].load((const T*)p.up + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + 256u * u, r = div_by(min(i, p.eights - 1), p.per);
        const int bg = block_byte(g[u]), bw = block_byte(w[u]);
        if (i >= p.eights) continue;   // four lanes of a block pass together
        float h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = gate_of<GELU>(g[u].get(j)).f * w[u].get(j);
        store8((H*)p.h + (size_t)i * 8, h);
        const size_t cg = (size_t)i + (size_t)r * p.per.d, cw = cg + p.per.d;   // eights of [m, 2 n]
        *(i32x2*)(p.codes + cg * 8) = encode8(g[u], bg);
        *(i32x2*)(p.codes + cw * 8) = encode8(w[u], bw);
        if ((i & 3) == 0) { p.scale[cg >> 2] = (uint8_t)bg; p.scale[cw >> 2] = (uint8_t)bw; }
    }
}

struct GatedGradArgs {
    const void* dh;
    const uint8_t* codes;
    const uint8_t* scale;
    void* dgate;
    void* dup;
    void* h;
    uint32_t eights;
    Divisor per;
    int64_t stride;
};
template <typename T, typename O, bool GELU, int U>
__global__ __launch_bounds__(256) void gated_grad(GatedGradArgs p) {
    const uint32_t i0 = blockIdx.x * (256u * U) + threadIdx.x;
    Eight<T> d[U];
    i32x2 cg[U], cw[U];
    int bg[U], bw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = min(i0 + 256u * u, p.eights - 1), r = div_by(i, p.per);
        d[u].load((const T*)p.dh + (size_t)i * 8);
        const size_t at = (size_t)i + (size_t)r * p.per.d;
        cg[u] = __builtin_nontemporal_load((const i32x2*)(p.codes + at * 8));
        cw[u] = __builtin_nontemporal_load((const i32x2*)(p.codes + (at + p.per.d) * 8));
        bg[u] = p.scale[at >> 2];
        bw[u] = p.scale[(at + p.per.d) >> 2];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + 256u * u;
        if (i >= p.eights) continue;
        const uint32_t r = div_by(i, p.per);
        float g[8], w[8], dg[8], dw[8], h[8];
        decode8(cg[u], bg[u], g);
        decode8(cw[u], bw[u], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Gate a = gate_of<GELU>(g[j]);
            const float dh = d[u].get(j);
            dg[j] = dh * w[j] * a.d;
            dw[j] = dh * a.f;
            h[j] = a.f * w[j];
        }
        const int64_t at = (int64_t)r * p.stride + (int64_t)(i - r * p.per.d) * 8;
        store8((O*)p.dgate + at, dg);
        store8((O*)p.dup + at, dw);
        if (p.h) store8((O*)p.h + (size_t)i * 8, h);
    }
}

}  // namespace fp8

// Eights a lane that the conversions of rows have on their way (16384 rows of 5120 bf16 values to 8 bits and back: 80 us with
// one, 78 with two or four).  The gated unit's lanes load two or three arrays and take one eight.
constexpr int kU = 2;
static uint32_t fp8_blocks(uint32_t eights, int u) { return (eights + 256u * u - 1) / (256u * u); }

hipError_t launch_fp8_quantize(const void* x, bool bf16, int64_t rows, int64_t k, int64_t stride, uint8_t* codes, uint8_t* scale,
                               hipStream_t s) {
    const uint32_t n = (uint32_t)(rows * k / 8);
    if (n == 0) return hipSuccess;
    const fp8::Divisor per = fp8::divisor((uint32_t)(k / 8));
    const dim3 grid(fp8_blocks(n, kU)), nt(256);
    const bool dense = stride == k || rows == 1;
    if (bf16) {
        if (dense) hipLaunchKernelGGL((fp8::quantize<uint16_t, true, kU>), grid, nt, 0, s, (const uint16_t*)x, n, per, stride, codes, scale);
        else hipLaunchKernelGGL((fp8::quantize<uint16_t, false, kU>), grid, nt, 0, s, (const uint16_t*)x, n, per, stride, codes, scale);
    } else {
        if (dense) hipLaunchKernelGGL((fp8::quantize<float, true, kU>), grid, nt, 0, s, (const float*)x, n, per, stride, codes, scale);
        else hipLaunchKernelGGL((fp8::quantize<float, false, kU>), grid, nt, 0, s, (const float*)x, n, per, stride, codes, scale);
    }
    return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const uint8_t* scale, int64_t rows, int64_t k, void* out, bool out_bf16,
                                 hipStream_t s) {
    const uint32_t n = (uint32_t)(rows * k / 8);
    if (n == 0) return hipSuccess;
    const dim3 grid(fp8_blocks(n, kU)), nt(256);
    if (out_bf16) hipLaunchKernelGGL((fp8::dequantize<uint16_t, kU>), grid, nt, 0, s, codes, scale, n, (uint16_t*)out);
    else hipLaunchKernelGGL((fp8::dequantize<float, kU>), grid, nt, 0, s, codes, scale, n, (float*)out);
    return hipGetLastError();
}

template <typename T, typename H>
static void launch_gated_t(const fp8::GatedArgs& p, bool gelu, hipStream_t s) {
    const dim3 grid(fp8_blocks(p.eights, 1)), nt(256);
    if (gelu) hipLaunchKernelGGL((fp8::gated<T, H, true, 1>), grid, nt, 0, s, p);
    else hipLaunchKernelGGL((fp8::gated<T, H, false, 1>), grid, nt, 0, s, p);
}

hipError_t launch_gated_act(const GatedActArgs& a, hipStream_t s) {
    const uint32_t n = (uint32_t)(a.m * a.n / 8);
    if (n == 0) return hipSuccess;
    const fp8::GatedArgs p{a.gate, a.up, a.h, a.codes, a.scale, n, fp8::divisor((uint32_t)(a.n / 8)), a.stride};
    if (a.bf16) {
        if (a.out_bf16) launch_gated_t<uint16_t, uint16_t>(p, a.gelu, s);
        else launch_gated_t<uint16_t, float>(p, a.gelu, s);
    } else {
        if (a.out_bf16) launch_gated_t<float, uint16_t>(p, a.gelu, s);
        else launch_gated_t<float, float>(p, a.gelu, s);
    }
    return hipGetLastError();
}

template <typename T, typename O>
static void launch_gated_grad_t(const fp8::GatedGradArgs& p, bool gelu, hipStream_t s) {
    const dim3 grid(fp8_blocks(p.eights, 1)), nt(256);
    if (gelu) hipLaunchKernelGGL((fp8::gated_grad<T, O, true, 1>), grid, nt, 0, s, p);
    else hipLaunchKernelGGL((fp8::gated_grad<T, O, false, 1>), grid, nt, 0, s, p);
}

hipError_t launch_gated_act_grad(const GatedActGradArgs& a, hipStream_t s) {
    const uint32_t n = (uint32_t)(a.m * a.n / 8);
    if (n == 0) return hipSuccess;
    const fp8::GatedGradArgs p{a.dh, a.codes, a.scale, a.dgate, a.dup, a.h, n, fp8::divisor((uint32_t)(a.n / 8)), a.stride};
    if (a.bf16) {
        if (a.out_bf16) launch_gated_grad_t<uint16_t, uint16_t>(p, a.gelu, s);
        else launch_gated_grad_t<uint16_t, float>(p, a.gelu, s);
    } else {
        if (a.out_bf16) launch_gated_grad_t<float, uint16_t>(p, a.gelu, s);
        else launch_gated_grad_t<float, float>(p, a.gelu, s);
    }
    return hipGetLastError();
}

}  // namespace gg
