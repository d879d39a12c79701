// abi_driver_lora.cpp -- the host-side argument checks of the low-rank adapters, of the 8-bit activation checkpoints and of
// the weight gradient from 8-bit rows under AddressSanitizer and UndefinedBehaviorSanitizer (api.hip and the launchers'
// arithmetic built with host instrumentation).  A few refused arguments with their codes, and a deterministic stream of
// random ones, sizes near 2^24, 2^31 and 2^63 among them, whose products the checks form before they refuse.  Runs only where
// no GPU is visible: a call that passed validation then fails at its first runtime call, so no fake address ever reaches a
// kernel.  Exit status 0 on success.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "groupgemm.h"

static int failures = 0;
#define EXPECT(call, code)                                                                    \
    do {                                                                                      \
        const int got_ = (int)(call);                                                         \
        if (got_ != (code)) {                                                                 \
            fprintf(stderr, "line %d: %s returned %d, expected %d\n", __LINE__, #call, got_, (code)); \
            ++failures;                                                                       \
        }                                                                                     \
    } while (0)

static uint64_t state = 0x2545F4914F6CDD1Dull;
static uint64_t next_u64() {   // splitmix64
    uint64_t z = (state += 0x9E3779B97F4A7C15ull);
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
static int64_t dim() {
    static const int64_t v[] = {-((int64_t)1 << 40), -32, -1, 0, 1, 7, 32, 96, 256, 4096, 14336, 65535, (1 << 24) - 1, 1 << 24, 1 << 27, 1 << 30,
                                INT32_MAX - 31, INT32_MAX, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX - 31, INT64_MAX};
    return v[next_u64() % (sizeof v / sizeof v[0])];
}
static int64_t small() { return (int64_t)(next_u64() % 700); }
static int64_t size() { return next_u64() % 2 ? dim() : 32 * small(); }
template <typename T = uint8_t> static T* ptr() {
    static const uintptr_t v[] = {0, 0x10000, 0x10001, 0x10002, 0x10008, 0x20000, (uintptr_t)1 << 44, (uintptr_t)2 << 44, (uintptr_t)3 << 44,
                                  (uintptr_t)4 << 44, (uintptr_t)5 << 44, (uintptr_t)6 << 44, (uintptr_t)7 << 44};
    return (T*)v[next_u64() % (sizeof v / sizeof v[0])];
}
static int code(int lo, int hi) { return lo + (int)(next_u64() % (uint64_t)(hi - lo + 1)); }
static gg_dtype type() { return (gg_dtype)code(next_u64() % 8 ? 0 : -1, next_u64() % 8 ? 2 : 4); }

int main() {
    int devices = 0;
    if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {
        printf("a GPU is visible: skipped (this driver passes fake addresses)\n");
        return 77;
    }
    uint8_t* far[10];
    for (int i = 0; i < 10; ++i) far[i] = (uint8_t*)((uintptr_t)(i + 1) << 44);
    const int64_t big = INT64_MAX;
    const gg_dtype BF = GG_DT_BF16;
    EXPECT(mxfp8_quantize(far[0], far[1], far[2], big, 32, 32, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp8_quantize(far[0], far[1], far[2], 4, 32, big, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp8_dequantize(far[0], far[1], far[2], INT32_MAX, INT32_MAX - 31, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(gated_act_mxfp8(far[0], far[1], far[2], far[3], far[4], 4, (int64_t)1 << 30, (int64_t)1 << 30, GG_ACT_SILU, BF, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(ragged_lora(far[0], far[1], far[2], (int32_t*)far[3], nullptr, nullptr, nullptr, far[4], nullptr, big, 32, 32, 4, 2, 32, 32, 32, BF, BF,
                       far[5], SIZE_MAX, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(ragged_lora(far[0], far[1], far[2], (int32_t*)far[3], nullptr, nullptr, nullptr, far[4], nullptr, 1 << 30, 32, 32, 4, 2, 32, 32, 32, BF, BF,
                       far[5], SIZE_MAX / 2, nullptr), GG_ERR_BAD_SHAPE);
    for (int i = 0; i < 400000; ++i) {
        const int64_t m = size(), k = size(), n = size();
        const int32_t g = next_u64() % 4 ? code(1, 64) : code(-2, 1100), r = next_u64() % 4 ? code(1, 64) : code(-2, 300);
        const size_t wsb = next_u64() % 4 ? SIZE_MAX / 2 : (size_t)next_u64() % 100000;
        switch (i % 8) {
            case 0: (void)mxfp8_quantize(ptr(), ptr(), ptr(), m, k, next_u64() % 2 ? k : dim(), type(), nullptr); break;
            case 1: (void)mxfp8_dequantize(ptr(), ptr(), ptr(), m, k, type(), nullptr); break;
            case 2: (void)gated_act_mxfp8(ptr(), ptr(), ptr(), ptr(), ptr(), m, n, next_u64() % 2 ? n : dim(), (gg_activation)code(-1, 2), type(), type(), nullptr); break;
            case 3: (void)gated_act_mxfp8_grad(ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), m, n, next_u64() % 2 ? n : dim(), (gg_activation)code(0, 1), type(), type(), nullptr); break;
            case 4: (void)ragged_dot_k_mxfp8(ptr(), ptr(), ptr(), ptr<int32_t>(), ptr(), m, k, n, g, type(), 1.f, 0.f, ptr(), wsb, nullptr); break;
            case 5: (void)ragged_lora(ptr(), ptr(), ptr(), ptr<int32_t>(), next_u64() % 2 ? nullptr : ptr<int32_t>(), ptr<float>(), ptr(), ptr(), ptr<float>(), m, k, n, r, g,
                                      next_u64() % 2 ? k : dim(), next_u64() % 2 ? n : dim(), next_u64() % 2 ? n : dim(), type(), type(), ptr(), wsb, nullptr); break;
            case 6: (void)ragged_lora_grad(ptr(), next_u64() % 2 ? nullptr : ptr(), ptr<float>(), ptr(), ptr(), ptr(), ptr<int32_t>(), ptr<float>(), ptr(), ptr(), ptr(), ptr(),
                                           m, k, n, r, g, type(), type(), type(), ptr(), wsb, nullptr); break;
            default: (void)gg_workspace_bytes((gg_op)code(0, 7), m, k, n, g, next_u64() % 2 ? r : dim(), type()); break;
        }
    }
    printf("%d failures\n", failures);
    return failures ? 1 : 0;
}
