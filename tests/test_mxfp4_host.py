"""Host checks of the MXFP4 and MoE-gradient entry points (CPU): every call below fails validation, so no
pointer is dereferenced."""
import ctypes

import pytest
import torch

from group_gemm_amd import _binding as B

P, ODD, A8 = 0x10000, 0x10001, 0x10008
OK, NULL_PTR, BAD_SHAPE, BAD_DTYPE, MISALIGNED, WS_SMALL, UNSUPPORTED = range(7)


def quantize(x=P, q=P, s=P, rows=4, k=64, stride=64, dt=1):
    return B.lib().mxfp4_quantize(x, q, s, rows, k, stride, dt, None)


def weights(w=P, q=P, s=P, g=2, k=64, n=16, dt=1):
    return B.lib().mxfp4_quantize_weights(w, q, s, g, k, n, dt, None)


def dequantize(q=P, s=P, out=P, g=2, n=16, k=64, dt=1):
    return B.lib().mxfp4_dequantize(q, s, out, g, n, k, dt, None)


def product(lhs=P, rhs=P, gs=P, out=P, m=8, k=64, n=16, g=2, dt=1, ls=P, rs=P, ws=P, wsb=4096):
    return B.lib().ragged_dot_m_mxfp4(lhs, rhs, gs, out, m, k, n, g, dt, ls, rs, ws, wsb, None)


def test_quantize():
    for a in ("x", "q", "s"):
        assert quantize(**{a: None}) == NULL_PTR
    assert quantize(rows=-1) == quantize(k=-32) == quantize(stride=63) == quantize(rows=1 << 31) == BAD_SHAPE
    assert quantize(rows=1 << 30, k=1024, stride=1024) == BAD_SHAPE   # too many (row, panel) pairs
    assert quantize(dt=2) == quantize(dt=3) == quantize(dt=9) == BAD_DTYPE
    assert quantize(k=48) == UNSUPPORTED
    assert quantize(x=ODD) == quantize(q=A8) == quantize(s=0x10004) == quantize(x=0x10002, dt=0) == MISALIGNED
    assert quantize(rows=0, x=None, q=None, s=None) == OK


def test_quantize_weights():
    for a in ("w", "q", "s"):
        assert weights(**{a: None}) == NULL_PTR
    assert weights(g=0) == weights(g=1025) == weights(n=-1) == weights(k=1 << 31) == BAD_SHAPE
    assert weights(n=1 << 30, k=1024) == BAD_SHAPE
    assert weights(dt=2) == weights(dt=-1) == BAD_DTYPE
    assert weights(k=40) == UNSUPPORTED
    assert weights(w=ODD) == weights(q=A8) == weights(s=0x10004) == MISALIGNED
    assert weights(n=0, w=None, q=None, s=None) == OK


def test_dequantize():
    for a in ("q", "s", "out"):
        assert dequantize(**{a: None}) == NULL_PTR
    assert dequantize(g=0) == dequantize(n=-1) == dequantize(n=1 << 30, k=1024) == BAD_SHAPE
    assert dequantize(dt=2) == dequantize(dt=3) == BAD_DTYPE
    assert dequantize(k=16) == UNSUPPORTED
    assert dequantize(out=ODD) == dequantize(q=A8) == dequantize(s=0x10004) == MISALIGNED
    assert dequantize(k=0, q=None, s=None, out=None) == OK


def test_product():
    for a in ("lhs", "rhs", "gs", "out", "ls", "rs", "ws"):
        assert product(**{a: None}) == NULL_PTR
    assert product(g=0) == product(g=1025) == product(m=-1) == product(n=1 << 31) == BAD_SHAPE
    assert product(m=(1 << 31) - 1, n=(1 << 31) - 1) == BAD_SHAPE        # more tiles than a launch holds
    assert product(dt=2) == product(dt=3) == BAD_DTYPE
    assert product(k=80) == UNSUPPORTED
    assert product(lhs=A8) == product(rhs=A8) == product(ls=0x10004) == product(rs=0x10004) == MISALIGNED
    assert product(out=ODD) == product(out=0x10002, dt=0) == product(ws=A8) == product(gs=0x10002) == MISALIGNED
    assert product(wsb=16) == WS_SMALL


def test_product_offsets_stay_in_32_bits():
    # 128 rows of codes have to stay below 2^31 bytes, column indices past n in 32 bits
    assert product(k=1 << 25) == product(k=(1 << 30)) == BAD_SHAPE
    assert product(m=1, n=(1 << 31) - 200) == BAD_SHAPE


def test_workspace_bytes():
    assert B.workspace_bytes("ragged_m", 8, 64, 16, 2, 0, B.FP4) > 0
    assert B.workspace_bytes("permute", 8, 64, 0, 2, 0, B.FP4) > 0
    for op in ("ragged_k", "padded_m", "padded_k"):
        assert B.workspace_bytes(op, 8, 64, 16, 2, 8, B.FP4) == 0


def test_other_products_refuse_e2m1():
    L = B.lib()
    assert L.ragged_dot_m(P, P, P, P, 8, 64, 16, 2, 3, 1, P, P, P, 4096, None) == BAD_DTYPE
    assert L.ragged_dot_m_nk(P, P, P, P, 8, 64, 16, 2, 3, 1, P, 4096, None) == UNSUPPORTED
    assert L.ragged_dot_k(P, P, P, P, 8, 64, 16, 2, 3, 0, P, 4096, None) == BAD_DTYPE
    assert L.padded_dot(2, P, P, P, P, 8, 64, 16, 2, 8, 3, 1, P, P, P, 1 << 20, None) == BAD_DTYPE


def test_permute_of_e2m1_rows():
    def permute(x=P, xs=P, e=P, sx=P, ss=P, gs=P, s2c=P, c2s=P, tokens=8, top_k=2, k=64, g=4, ws=P, wsb=1 << 20):
        return B.lib().moe_permute(x, xs, e, sx, ss, gs, s2c, c2s, tokens, top_k, k, g, 3, ws, wsb, None)
    assert permute(xs=None) == permute(ss=None) == permute(x=None) == NULL_PTR
    assert permute(k=48) == UNSUPPORTED
    assert permute(xs=0x10004) == permute(ss=0x10004) == MISALIGNED
    assert permute(k=256 * 65536) == BAD_SHAPE   # more panels than a launch holds
    assert permute(wsb=8) == WS_SMALL


def test_permute_grad():
    def grad(d=P, c=P, dx=P, tokens=4, top_k=2, k=8, i=1, o=1):
        return B.lib().moe_permute_grad(d, c, dx, tokens, top_k, k, i, o, None)
    for a in ("d", "c", "dx"):
        assert grad(**{a: None}) == NULL_PTR
    assert grad(tokens=-1) == grad(top_k=0) == grad(k=-1) == grad(tokens=1 << 30) == BAD_SHAPE
    assert grad(i=2) == grad(o=3) == BAD_DTYPE
    assert grad(d=ODD) == grad(c=0x10002) == grad(dx=0x10002, o=0) == MISALIGNED
    assert grad(tokens=0, d=None, c=None, dx=None) == OK


def test_unpermute_grad():
    def grad(dout=P, y=P, c=P, s=P, w=P, dy=P, dw=P, tokens=4, top_k=2, n=8, dt=1):
        return B.lib().moe_unpermute_grad(dout, y, c, s, w, dy, dw, tokens, top_k, n, dt, None)
    for a in ("dout", "y", "c", "s", "w", "dy", "dw"):
        assert grad(**{a: None}) == NULL_PTR
    assert grad(tokens=-1) == grad(top_k=0) == grad(n=-1) == grad(tokens=1 << 30) == BAD_SHAPE
    assert grad(dt=2) == grad(dt=3) == BAD_DTYPE
    assert grad(dout=ODD) == grad(y=ODD) == grad(dy=ODD) == grad(w=0x10002) == grad(dw=0x10002) == grad(s=0x10002) == MISALIGNED
    assert grad(tokens=0, dout=None, y=None, c=None, s=None, w=None, dy=None, dw=None) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    q = torch.zeros(8, 32, dtype=torch.uint8).view(B.FP4)
    s = torch.zeros(1, 8, 8, dtype=torch.uint8)
    i = torch.zeros(8, dtype=torch.int32)
    for call in (lambda: B.mxfp4_quantize(x),
                 lambda: B.mxfp4_quantize_weights(torch.zeros(2, 32, 8)),
                 lambda: B.mxfp4_dequantize(q, s),
                 lambda: B.ragged_dot_m_mxfp4(q, q[None], i[:1], s, s[None]),
                 lambda: B.moe_permute(q, torch.zeros(8, 2, dtype=torch.int32), 4, x_scale=s),
                 lambda: B.moe_permute_grad(x, i, 2),
                 lambda: B.moe_unpermute_grad(x[:4], x, i, i, torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_exported_names():
    import group_gemm_amd as G
    for name in ("mxfp4_quantize", "mxfp4_quantize_weights", "mxfp4_dequantize", "ragged_dot_m_mxfp4", "moe_permute_grad",
                 "moe_unpermute_grad"):
        assert callable(getattr(G, name))
        assert isinstance(getattr(B.lib(), name), ctypes._CFuncPtr)
