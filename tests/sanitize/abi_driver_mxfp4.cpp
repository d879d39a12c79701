// abi_driver_mxfp4.cpp -- the host-side argument checks of the MXFP4 calls and of the gradients of permute and
// un-permute under AddressSanitizer and UndefinedBehaviorSanitizer (api.hip and the launchers built with host
// instrumentation).  Refused arguments with the code that each must give, and a deterministic stream of random
// ones, sizes near 2^25, 2^30 and 2^31 among them, whose products the checks form before they refuse.  Runs only
// where no GPU is visible: a call that passed validation then fails at its first runtime call, so no fake address
// ever reaches a kernel.  Exit status 0 on success.
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

static uint64_t state = 0x9E3779B97F4A7C15ull;
static uint64_t next_u64() {   // splitmix64
    uint64_t z = (state += 0x9E3779B97F4A7C15ull);
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
static int64_t pick_dim() {
    static const int64_t v[] = {-((int64_t)1 << 40), -32, -1, 0, 1, 7, 8, 31, 32, 96, 256, 288, 4096, 14336, 65535, (1 << 24) - 1, 1 << 24,
                                1 << 25, (1 << 26) - 4, 1 << 26, 1 << 29, 1 << 30, INT32_MAX - 256, INT32_MAX - 31, INT32_MAX,
                                (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX - 255, INT64_MAX};
    return v[next_u64() % (sizeof v / sizeof v[0])];
}
template <typename T = uint8_t>
static T* pick_ptr() {
    static const uintptr_t v[] = {0,       0x10000, 0x10001, 0x10002, 0x10004, 0x10008, 0x10010, (uintptr_t)1 << 44, (uintptr_t)2 << 44,
                                  (uintptr_t)3 << 44, (uintptr_t)4 << 44};
    return (T*)v[next_u64() % (sizeof v / sizeof v[0])];
}
static int pick_code(int lo, int hi) { return lo + (int)(next_u64() % (uint64_t)(hi - lo + 1)); }

int main() {
    int devices = 0;
    if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {
        printf("a GPU is visible: skipped (this driver passes fake addresses)\n");
        return 77;
    }
    uint8_t* const P = (uint8_t*)0x10000;   // aligned, never dereferenced
    uint8_t* const ODD = (uint8_t*)0x10001;
    int32_t* const I = (int32_t*)P;
    float* const F = (float*)P;
    const gg_dtype BF = GG_DT_BF16, F32 = GG_DT_F32, E4 = GG_DT_E4M3, E2 = GG_DT_E2M1;
    const int64_t big = INT64_MAX;

    EXPECT(mxfp4_quantize(nullptr, P, P, 4, 64, 64, BF, nullptr), GG_ERR_NULL_PTR);
    EXPECT(mxfp4_quantize(P, P, P, 4, 64, 63, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp4_quantize(P, P, P, big, 64, 64, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp4_quantize(P, P, P, 4, 64, big, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp4_quantize(P, P, P, INT32_MAX, INT32_MAX - 31, INT32_MAX, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp4_quantize(P, P, P, 4, 64, 64, E2, nullptr), GG_ERR_BAD_DTYPE);
    EXPECT(mxfp4_quantize(P, P, P, 4, 48, 48, F32, nullptr), GG_ERR_UNSUPPORTED);
    EXPECT(mxfp4_quantize(ODD, P, P, 4, 64, 64, BF, nullptr), GG_ERR_MISALIGNED);
    EXPECT(mxfp4_quantize_weights(P, P, P, 0, 64, 16, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp4_quantize_weights(P, P, P, 1024, INT32_MAX - 31, INT32_MAX, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp4_quantize_weights(P, P, nullptr, 2, 64, 16, F32, nullptr), GG_ERR_NULL_PTR);
    EXPECT(mxfp4_quantize_weights(P, P, P, 2, 64, 16, E4, nullptr), GG_ERR_BAD_DTYPE);
    EXPECT(mxfp4_dequantize(P, P, P, 1025, 16, 64, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp4_dequantize(P, P, P, 1024, INT32_MAX, INT32_MAX - 31, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(mxfp4_dequantize(P, P, nullptr, 2, 16, 64, BF, nullptr), GG_ERR_NULL_PTR);
    EXPECT(mxfp4_dequantize(P, (uint8_t*)0x10004, P, 2, 16, 64, BF, nullptr), GG_ERR_MISALIGNED);

    EXPECT(ragged_dot_m_mxfp4(P, P, nullptr, P, 8, 64, 16, 2, BF, P, P, P, 4096, nullptr), GG_ERR_NULL_PTR);
    EXPECT(ragged_dot_m_mxfp4(P, P, I, P, 8, 64, 16, 2, E2, P, P, P, 4096, nullptr), GG_ERR_BAD_DTYPE);
    EXPECT(ragged_dot_m_mxfp4(P, P, I, P, 8, 80, 16, 2, BF, P, P, P, 4096, nullptr), GG_ERR_UNSUPPORTED);
    EXPECT(ragged_dot_m_mxfp4(P, P, I, P, 8, 64, 16, 2, BF, P, P, P, 8, nullptr), GG_ERR_WORKSPACE_TOO_SMALL);
    EXPECT(ragged_dot_m_mxfp4(P, P, I, P, INT32_MAX, 32, 1, 1, BF, P, P, P, 4096, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(ragged_dot_m_mxfp4(P, P, I, P, INT32_MAX, 32, INT32_MAX - 256, 1, BF, P, P, P, 4096, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(ragged_dot_m_mxfp4(P, P, I, P, 1, INT32_MAX - 31, 1, 1, BF, P, P, P, 4096, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(gg_mxfp4_kernel(8192, 4096, 14336, 8, 256), GG_FP4_TILE);
    EXPECT(gg_mxfp4_kernel(1, (1 << 25) - 32, 1, 1, 1), GG_FP4_BLOCK);
    EXPECT(gg_mxfp4_kernel(big, 32, 1, 1, 256), -1);

    const size_t need = gg_workspace_bytes(GG_OP_PERMUTE, 128, 64, 0, 8, 0, E2);
    EXPECT(need > 256, 1);
    EXPECT(moe_permute(P, nullptr, I, P, P, I, I, I, 64, 2, 64, 8, E2, P, need, nullptr), GG_ERR_NULL_PTR);
    EXPECT(moe_permute(P, P, I, P, (uint8_t*)0x10004, I, I, I, 64, 2, 64, 8, E2, P, need, nullptr), GG_ERR_MISALIGNED);
    EXPECT(moe_permute(P, P, I, P, P, I, I, I, 64, 2, 256 * 65536, 8, E2, P, need, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(moe_permute_grad(P, I, (uint8_t*)P + 512, 16, 2, 64, BF, BF, nullptr), GG_ERR_UNSUPPORTED);
    EXPECT(moe_permute_grad(P, I, nullptr, 16, 2, 64, BF, BF, nullptr), GG_ERR_NULL_PTR);
    EXPECT(moe_permute_grad(P, I, P, big, 2, 64, BF, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(moe_permute_grad((void*)(1ull << 46), (int32_t*)(2ull << 45), P, 1 << 30, 1, INT32_MAX, F32, F32, nullptr), GG_ERR_UNSUPPORTED);
    EXPECT(moe_unpermute_grad(P, P, I, I, F, P, F, 16, 2, 64, BF, nullptr), GG_ERR_UNSUPPORTED);
    EXPECT(moe_unpermute_grad(P, P, I, I, F, P, nullptr, 16, 2, 64, BF, nullptr), GG_ERR_NULL_PTR);
    EXPECT(moe_unpermute_grad(P, P, I, I, F, P, F, 16, 0, 64, BF, nullptr), GG_ERR_BAD_SHAPE);
    EXPECT(moe_unpermute_grad(P, P, I, I, (float*)0x10002, P, F, 16, 2, 64, BF, nullptr), GG_ERR_MISALIGNED);

    // random arguments: every call returns a status code and touches no memory it was handed
    long counts[8] = {};
    for (int it = 0; it < 200000; ++it) {
        const int64_t m = pick_dim(), k = pick_dim(), n = pick_dim();
        const int32_t g = (int32_t)pick_code(-2, 1100), top_k = next_u64() % 16 ? (int32_t)pick_code(-1, 9) : INT32_MAX;
        const gg_dtype in = (gg_dtype)pick_code(-1, 4), out = (gg_dtype)pick_code(-1, 4);
        const size_t wsb = (size_t)pick_code(0, 1 << 20);
        int rc;
        switch (it % 7) {
            case 0: rc = mxfp4_quantize(pick_ptr(), pick_ptr(), pick_ptr(), m, k, next_u64() % 2 ? k : pick_dim(), in, nullptr); break;
            case 1: rc = mxfp4_quantize_weights(pick_ptr(), pick_ptr(), pick_ptr(), g, k, n, in, nullptr); break;
            case 2: rc = mxfp4_dequantize(pick_ptr(), pick_ptr(), pick_ptr(), g, n, k, out, nullptr); break;
            case 3: rc = ragged_dot_m_mxfp4(pick_ptr(), pick_ptr(), pick_ptr<int32_t>(), pick_ptr(), m, k, n, g, out, pick_ptr(), pick_ptr(),
                                            pick_ptr(), wsb, nullptr); break;
            case 4: rc = moe_permute(pick_ptr(), pick_ptr(), pick_ptr<int32_t>(), pick_ptr(), pick_ptr(), pick_ptr<int32_t>(),
                                     pick_ptr<int32_t>(), pick_ptr<int32_t>(), m, top_k, k, g, GG_DT_E2M1, pick_ptr(), wsb, nullptr); break;
            case 5: rc = moe_permute_grad(pick_ptr(), pick_ptr<int32_t>(), pick_ptr(), m, top_k, k, in, out, nullptr); break;
            default: rc = moe_unpermute_grad(pick_ptr(), pick_ptr(), pick_ptr<int32_t>(), pick_ptr<int32_t>(), pick_ptr<float>(),
                                             pick_ptr(), pick_ptr<float>(), m, top_k, n, in, nullptr);
        }
        if (rc < 0 || rc > 7) { fprintf(stderr, "iteration %d: status %d out of range\n", it, rc); ++failures; }
        else ++counts[rc];
        const int which = gg_mxfp4_kernel(m, k, n, g, pick_code(-1, 512));
        if (which < -1 || which > 2) { fprintf(stderr, "iteration %d: kernel %d\n", it, which); ++failures; }
        (void)gg_workspace_bytes((gg_op)pick_code(-1, 5), m, k, n, g, pick_dim(), GG_DT_E2M1);
    }
    printf("statuses");
    for (long c : counts) printf(" %ld", c);
    printf("\nabi driver (mxfp4): %d failures\n", failures);
    return failures ? 2 : 0;
}
