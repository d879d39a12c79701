"""Shapes that need more workgroups than one launch holds (2^32 threads along x), or more rows than the kernels'
32-bit tile counts take, are refused as shapes before anything is launched (CPU).  Every call below fails
validation, so no pointer is dereferenced."""
from group_gemm_amd import _binding as B

BAD_SHAPE = 2
FAR = 1 << 44   # arrays this far apart do not overlap
PTRS = [FAR * i for i in range(1, 9)]


def test_product_rows():
    def product(m, n=1, g=1, k=32):
        lhs, rhs, gs, out, ls, rs, ws, _ = PTRS
        return B.lib().ragged_dot_m_mxfp4(lhs, rhs, gs, out, m, k, n, g, 1, ls, rs, ws, 4096, None)
    # one group: the rows rounded up to whole tiles would pass 2^31
    assert product((1 << 31) - 1) == product((1 << 31) - 60) == product((1 << 31) - 64, g=7) == BAD_SHAPE
    assert product(1 << 30) == product(1 << 30, g=1024) == BAD_SHAPE


def test_quantisation():
    x, q, s = PTRS[:3]
    L = B.lib()
    assert L.mxfp4_quantize(x, q, s, 1 << 29, 32, 32, 1, None) == BAD_SHAPE           # 32 rows a workgroup
    assert L.mxfp4_quantize(x, q, s, (1 << 30) - 1, 256, 256, 0, None) == BAD_SHAPE
    assert L.mxfp4_quantize_weights(x, q, s, 1024, 256 << 14, 1, 1, None) == BAD_SHAPE   # a workgroup a panel and group
    assert L.mxfp4_dequantize(q, s, x, 1024, 1, 256 << 14, 1, None) == BAD_SHAPE
    assert L.mxfp4_dequantize(q, s, x, 1, 1 << 29, 32, 1, None) == BAD_SHAPE


def test_permute_and_back():
    L = B.lib()
    x, xs, e, sx, ss, gs, i, ws = PTRS
    for dtype, scale, sorted_scale in ((1, None, None), (3, xs, ss)):
        assert L.moe_permute(x, scale, e, sx, sorted_scale, gs, i, i, 1 << 25, 2, 32, 8, dtype, ws, 1 << 40, None) == BAD_SHAPE
    assert L.moe_unpermute(x, i, xs, sx, 1 << 25, 1, 520, 1, 1, None) == BAD_SHAPE    # two tokens a workgroup
    assert L.moe_unpermute(x, i, xs, sx, 1 << 26, 1, 8, 1, 1, None) == BAD_SHAPE      # four
    assert L.moe_permute_grad(x, i, sx, 1 << 25, 1, 520, 1, 1, None) == BAD_SHAPE
    assert L.moe_permute_grad(x, i, sx, 1 << 26, 2, 8, 0, 1, None) == BAD_SHAPE
    assert L.moe_unpermute_grad(x, sx, i, e, xs, ss, gs, 1 << 25, 1, 520, 1, None) == BAD_SHAPE
    assert L.moe_unpermute_grad(x, sx, i, e, xs, ss, gs, 1 << 26, 2, 8, 1, None) == BAD_SHAPE
