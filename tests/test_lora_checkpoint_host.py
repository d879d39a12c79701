"""Host checks of the adapters' and the 8-bit checkpoints' entry points (CPU): every call below fails validation or has
nothing to do, so no pointer is dereferenced."""
import pytest
import torch

from group_gemm_amd import _binding as B

OK, NULL_PTR, BAD_SHAPE, BAD_DTYPE, MISALIGNED, WS_SMALL, UNSUPPORTED = range(7)
F32, BF16, E4M3, E2M1 = 0, 1, 2, 3
A, STEP = 0x1000000, 0x1000000          # made-up addresses, far apart


def at(i, off=0):
    return A + STEP * i + off


def quantize(x=at(0), q=at(1), s=at(2), rows=4, k=64, stride=64, dt=BF16):
    return B.lib().mxfp8_quantize(x, q, s, rows, k, stride, dt, None)


def dequantize(q=at(0), s=at(1), out=at(2), rows=4, k=64, dt=BF16):
    return B.lib().mxfp8_dequantize(q, s, out, rows, k, dt, None)


def gated(gate=at(0), up=at(1), h=at(2), q=at(3), s=at(4), m=4, n=64, stride=64, act=0, dt=BF16, odt=BF16):
    return B.lib().gated_act_mxfp8(gate, up, h, q, s, m, n, stride, act, dt, odt, None)


def gated_grad(dh=at(0), q=at(1), s=at(2), dgate=at(3), dup=at(4), h=at(5), m=4, n=64, stride=64, act=0, dt=BF16, odt=BF16):
    return B.lib().gated_act_mxfp8_grad(dh, q, s, dgate, dup, h, m, n, stride, act, dt, odt, None)


def wgrad(lhs=at(0), ls=at(1), dout=at(2), gs=at(3), out=at(4), m=8, k=64, n=16, g=2, odt=F32, ws=at(5), wsb=4096):
    return B.lib().ragged_dot_k_mxfp8(lhs, ls, dout, gs, out, m, k, n, g, odt, 1.0, 0.0, ws, wsb, None)


def lora(x=at(0), a=at(1), b=at(2), gs=at(3), rg=None, sc=at(5), base=at(6), out=at(7), v=at(8), m=8, k=64, n=16, r=4, g=2, xs=64, bs=16, os=16,
         dt=BF16, odt=BF16, ws=at(9), wsb=1 << 20):
    return B.lib().ragged_lora(x, a, b, gs, rg, sc, base, out, v, m, k, n, r, g, xs, bs, os, dt, odt, ws, wsb, None)


def lora_grad(x=at(0), xs=None, v=at(1), dout=at(2), a=at(3), b=at(4), gs=at(5), sc=at(6), dbase=at(7), dx=at(8), da=at(9), db=at(10), m=8, k=64,
              n=16, r=4, g=2, xdt=BF16, dt=BF16, gdt=F32, ws=at(11), wsb=1 << 22):
    return B.lib().ragged_lora_grad(x, xs, v, dout, a, b, gs, sc, dbase, dx, da, db, m, k, n, r, g, xdt, dt, gdt, ws, wsb, None)


def test_quantize():
    for name in ("x", "q", "s"):
        assert quantize(**{name: None}) == NULL_PTR
    assert quantize(rows=-1) == quantize(k=-32) == quantize(stride=63) == quantize(rows=1 << 31) == quantize(stride=1 << 32) == BAD_SHAPE
    assert quantize(rows=1 << 28, k=64) == BAD_SHAPE                # 2^34 elements
    assert quantize(dt=E4M3) == quantize(dt=9) == quantize(dt=-1) == BAD_DTYPE
    assert quantize(k=48) == UNSUPPORTED
    assert quantize(x=at(0, 1)) == quantize(q=at(1, 8)) == quantize(x=at(0, 2), dt=F32) == MISALIGNED
    assert quantize(q=at(0)) == quantize(s=at(0, 511)) == quantize(s=at(1, 255)) == UNSUPPORTED
    assert quantize(rows=0, x=None, q=None, s=None) == OK


def test_dequantize():
    for name in ("q", "s", "out"):
        assert dequantize(**{name: None}) == NULL_PTR
    assert dequantize(rows=-1) == dequantize(k=1 << 31) == dequantize(rows=1 << 28) == BAD_SHAPE
    assert dequantize(dt=E4M3) == BAD_DTYPE
    assert dequantize(k=16) == UNSUPPORTED
    assert dequantize(q=at(0, 4)) == dequantize(out=at(2, 1)) == MISALIGNED
    assert dequantize(out=at(0)) == dequantize(out=at(1)) == UNSUPPORTED
    assert dequantize(k=0, q=None, s=None, out=None) == OK


def test_gated():
    for name in ("gate", "up", "h", "q", "s"):
        assert gated(**{name: None}) == NULL_PTR
    assert gated(m=-1) == gated(n=-32) == gated(stride=32) == gated(n=1 << 31) == gated(m=1 << 27, n=64) == BAD_SHAPE   # 2 n a row
    assert gated(n=(1 << 30) + 32, m=1, stride=(1 << 30) + 32) == BAD_SHAPE
    assert gated(dt=E4M3) == gated(odt=E2M1) == BAD_DTYPE
    assert gated(n=40) == gated(act=2) == gated(act=-1) == UNSUPPORTED
    assert gated(gate=at(0, 1)) == gated(up=at(1, 1)) == gated(h=at(2, 2), odt=F32) == gated(q=at(3, 8)) == MISALIGNED
    assert gated(h=at(0)) == gated(h=at(1, 64)) == gated(q=at(0)) == gated(s=at(1)) == gated(s=at(3, 16)) == gated(h=at(3)) == UNSUPPORTED
    assert gated(h=at(0, 128), stride=127) == UNSUPPORTED           # not a pitch of rows that lie between gate's
    assert gated(m=0, gate=None, up=None, h=None, q=None, s=None) == OK


def test_gated_grad():
    for name in ("dh", "q", "s", "dgate", "dup"):
        assert gated_grad(**{name: None}) == NULL_PTR
    assert gated_grad(m=-1) == gated_grad(stride=63) == gated_grad(m=1 << 27) == BAD_SHAPE
    assert gated_grad(dt=E4M3) == gated_grad(odt=5) == BAD_DTYPE
    assert gated_grad(n=16, stride=16) == gated_grad(act=7) == UNSUPPORTED
    assert gated_grad(dh=at(0, 1)) == gated_grad(dup=at(4, 1)) == gated_grad(h=at(5, 1)) == gated_grad(q=at(1, 1)) == MISALIGNED
    for name in ("dgate", "dup", "h"):
        assert gated_grad(**{name: at(0, 2)}) == UNSUPPORTED        # in dh, but not dh
        assert gated_grad(**{name: at(0), "odt": F32}) == UNSUPPORTED
        assert gated_grad(**{name: at(1)}) == gated_grad(**{name: at(2)}) == UNSUPPORTED
    assert gated_grad(dgate=at(0), stride=128) == UNSUPPORTED
    assert gated_grad(dgate=at(4)) == gated_grad(h=at(3)) == gated_grad(h=at(4)) == gated_grad(dgate=at(0), h=at(0)) == UNSUPPORTED
    assert gated_grad(dgate=at(3), dup=at(3, 64), stride=128) == UNSUPPORTED   # halves of 64 bf16 begin 128 bytes apart
    assert gated_grad(n=0, stride=0, dh=None, q=None, s=None, dgate=None, dup=None, h=None) == OK


def test_weight_gradient():
    for name in ("lhs", "ls", "dout", "gs", "out", "ws"):
        assert wgrad(**{name: None}) == NULL_PTR
    assert wgrad(g=0) == wgrad(g=1025) == wgrad(m=-1) == wgrad(n=1 << 31) == BAD_SHAPE
    assert wgrad(odt=E4M3) == BAD_DTYPE
    assert wgrad(k=48) == UNSUPPORTED
    assert wgrad(lhs=at(0, 8)) == wgrad(dout=at(2, 1)) == wgrad(out=at(4, 2)) == wgrad(ws=at(5, 8)) == wgrad(gs=at(3, 2)) == MISALIGNED
    assert wgrad(wsb=16) == WS_SMALL


def test_lora():
    for name in ("x", "a", "b", "out", "ws"):
        assert lora(**{name: None}) == NULL_PTR
    assert lora(gs=None) == NULL_PTR and lora(rg=at(4)) == UNSUPPORTED   # neither, both
    assert lora(g=0) == lora(g=1025) == lora(m=-1) == lora(n=1 << 31) == lora(r=0) == lora(r=257) == BAD_SHAPE
    assert lora(xs=63) == lora(bs=15) == lora(os=15) == lora(xs=1 << 32) == BAD_SHAPE
    assert lora(dt=E4M3) == lora(odt=E4M3) == lora(dt=E2M1) == BAD_DTYPE
    assert lora(x=at(0, 1)) == lora(a=at(1, 1)) == lora(b=at(2, 1)) == lora(gs=at(3, 2)) == lora(sc=at(5, 2)) == MISALIGNED
    assert lora(base=at(6, 1)) == lora(out=at(7, 2), odt=F32) == lora(v=at(8, 2)) == lora(ws=at(9, 8)) == MISALIGNED
    assert lora(wsb=256) == WS_SMALL
    for name in ("x", "a", "b", "gs", "sc", "v", "ws"):
        i = dict(x=0, a=1, b=2, gs=3, sc=5, v=8, ws=9)[name]
        assert lora(out=at(i)) == UNSUPPORTED, name
    for i in (0, 1, 2, 3, 5, 6, 7, 9):
        assert lora(v=at(i)) == UNSUPPORTED
    for i in (0, 1, 2, 3, 5, 6):
        assert lora(ws=at(i)) == UNSUPPORTED
    assert lora(gs=None, rg=at(4), out=at(4)) == UNSUPPORTED
    assert lora(out=at(6, 2)) == lora(out=at(6), os=32) == UNSUPPORTED   # in base, but not base
    assert lora(out=at(6, 16), os=32, bs=32) == UNSUPPORTED              # rows that share half their columns
    assert lora(m=0, x=None, a=None, b=None, base=None, out=None, v=None) == OK


def test_lora_grad():
    for name in ("x", "v", "dout", "a", "b", "gs", "da", "db", "ws"):
        assert lora_grad(**{name: None}) == NULL_PTR
    assert lora_grad(dx=None) == NULL_PTR                                # dbase without dx
    assert lora_grad(xdt=E4M3) == NULL_PTR                               # codes without scales
    assert lora_grad(g=0) == lora_grad(m=-1) == lora_grad(k=1 << 31) == lora_grad(r=0) == lora_grad(r=300) == BAD_SHAPE
    assert lora_grad(xdt=F32) == lora_grad(xdt=E4M3, xs=at(12), dt=F32) == lora_grad(dt=E4M3) == lora_grad(gdt=E4M3) == BAD_DTYPE
    assert lora_grad(xs=at(12)) == BAD_DTYPE                             # scales without codes
    assert lora_grad(xdt=E4M3, xs=at(12), k=48) == UNSUPPORTED
    assert lora_grad(xdt=E4M3, xs=at(12), x=at(0, 8)) == lora_grad(v=at(1, 2)) == lora_grad(da=at(9, 2)) == lora_grad(ws=at(11, 8)) == MISALIGNED
    assert lora_grad(dout=at(2, 1)) == lora_grad(dx=at(8, 1)) == lora_grad(gs=at(5, 1)) == lora_grad(db=at(10, 2)) == MISALIGNED
    assert lora_grad(wsb=1024) == WS_SMALL
    for name in ("dx", "da", "db", "ws"):
        for i in (0, 1, 2, 3, 4, 5, 6):
            assert lora_grad(**{name: at(i)}) == UNSUPPORTED, (name, i)
    assert lora_grad(dx=at(7, 2)) == lora_grad(da=at(7)) == lora_grad(da=at(8)) == lora_grad(da=at(10)) == lora_grad(db=at(8)) == UNSUPPORTED
    assert lora_grad(ws=at(7)) == lora_grad(ws=at(8)) == lora_grad(ws=at(9)) == lora_grad(ws=at(10)) == UNSUPPORTED
    assert lora_grad(xdt=E4M3, xs=at(12), dx=at(12)) == UNSUPPORTED


def test_workspace_bytes():
    need = B.lib().gg_workspace_bytes
    assert need(5, 8, 64, 16, 2, 4, BF16) >= 256 + 8 * 4 * 4
    for op in (5, 6):
        assert need(op, 8, 64, 16, 2, 0, BF16) == need(op, 8, 64, 16, 2, 257, BF16) == need(op, 8, 64, 16, 0, 4, BF16) == 0
        assert need(op, 8, 64, 16, 2, 4, E4M3) == need(op, 1 << 31, 64, 16, 2, 4, BF16) == 0
    # the gradients': both weights with their axes swapped, u, and two parts a chunk of rows
    assert need(6, 0, 64, 16, 2, 4, F32) >= 256 + 2 * 4 * (64 + 16) * 4
    assert need(6, 4096, 4096, 4096, 8, 16, BF16) < 256 + 2 * 8 * 16 * 8192 + 34 * 4096 * 16 * 4 + 2 * 17 * 8192 * 16 * 4


def test_launch_limits():
    """Shapes that need more workgroups than a launch holds are refused before the first of a call's launches."""
    far = [(1 << 44) * i for i in range(1, 13)]
    L = B.lib()

    def lora_far(m, n, g, any_order):
        ids = (None, far[3]) if any_order else (far[3], None)
        return L.ragged_lora(far[0], far[1], far[2], *ids, None, far[4], far[5], None, m, 8, n, 4, g, 8, n, n, BF16, BF16, far[6], 1 << 43, None)

    def grad_far(m, k, n, g):
        return L.ragged_lora_grad(far[0], None, far[1], far[2], far[3], far[4], far[5], None, None, far[6], far[7], far[8], m, k, n, 4, g, BF16, BF16, F32,
                                  far[9], 1 << 43, None)

    assert lora_far(1 << 28, 8, 1, False) == lora_far(1 << 27, 4096, 1, False) == lora_far(1 << 24, 1 << 16, 8, True) == BAD_SHAPE
    assert grad_far(1 << 28, 8, 8, 1) == grad_far(1, 1 << 28, 8, 1) == grad_far(1, 8, 1 << 20, 1024) == BAD_SHAPE


# the binding's own checks, with CPU tensors in the place of the GPU's

def no_call(monkeypatch):
    monkeypatch.setattr(B, "_call", lambda *a: pytest.fail("the call was not refused"))


@pytest.mark.parametrize("call", [
    lambda t: B.mxfp8_quantize(t(4, 64)), lambda t: B.mxfp8_dequantize(t(4, 64, dtype=torch.uint8), t(4, 2, dtype=torch.uint8)),
    lambda t: B.gated_act_mxfp8(t(4, 64), t(4, 64)),
    lambda t: B.gated_act_mxfp8_grad(t(4, 64), t(4, 128, dtype=torch.uint8), t(4, 4, dtype=torch.uint8)),
    lambda t: B.ragged_lora(t(4, 64), t(2, 3, 64), t(2, 5, 3), t(2, dtype=torch.int32)),
    lambda t: B.ragged_lora_grad(t(4, 64), t(4, 3), t(4, 5), t(2, 3, 64), t(2, 5, 3), t(2, dtype=torch.int32)),
    lambda t: B.ragged_dot_k(t(4, 64, dtype=torch.uint8), t(4, 8, dtype=torch.bfloat16), t(2, dtype=torch.int32), lhs_scale=t(4, 2, dtype=torch.uint8))])
def test_cpu_tensors_are_refused(call, monkeypatch):
    no_call(monkeypatch)
    with pytest.raises(ValueError, match="must be on a CUDA"):
        call(lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype))


def device_blind(monkeypatch):
    """The binding's checks of shapes and types on CPU tensors: only the device's are left out."""
    def tensor(t, name, device, shape=None, dtype=None, dtypes=None, contiguous=True):
        if torch.is_tensor(t) and contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape")
        if dtype is not None and t.dtype != dtype or dtypes is not None and t.dtype not in dtypes:
            raise ValueError(f"{name} has dtype")
    monkeypatch.setattr(B, "_tensor", tensor)
    no_call(monkeypatch)


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


U8, I32, BF = torch.uint8, torch.int32, torch.bfloat16
REFUSED = [
    (lambda: B.mxfp8_quantize(z(4, 48)), "k % 32"), (lambda: B.mxfp8_quantize(z(64, 4).t()), "unit column stride"),
    (lambda: B.mxfp8_quantize(z(1, 64).expand(4, 64)), "do not overlap"), (lambda: B.mxfp8_quantize(z(4, 64, dtype=torch.float16)), "dtype"),
    (lambda: B.mxfp8_quantize(z(4, 64), out=(z(4, 32, dtype=U8), None)), "codes has shape"),
    (lambda: B.mxfp8_dequantize(z(4, 64, dtype=U8), z(4, 3, dtype=U8)), "scale has shape"),
    (lambda: B.mxfp8_dequantize(z(4, 40, dtype=U8), z(4, 1, dtype=U8)), "k % 32"),
    (lambda: B.gated_act_mxfp8(z(4, 64), z(4, 128)[:, :64]), "one row stride"), (lambda: B.gated_act_mxfp8(z(4, 64), z(4, 64), act="relu"), "act must be"),
    (lambda: B.gated_act_mxfp8(z(4, 64), z(4, 32)), "up has shape"), (lambda: B.gated_act_mxfp8(z(4, 40), z(4, 40)), "n % 32"),
    (lambda: B.gated_act_mxfp8_grad(z(4, 64), z(4, 64, dtype=U8), z(4, 4, dtype=U8)), "codes has shape"),
    (lambda: B.gated_act_mxfp8_grad(z(4, 64), z(4, 128, dtype=U8), z(4, 4, dtype=U8), act=None), "act must be"),
    (lambda: B.gated_act_mxfp8_grad(z(4, 64), z(4, 128, dtype=U8), z(4, 4, dtype=U8), out=(z(4, 64), z(4, 128)[:, 64:], None)), "one row stride"),
    (lambda: B.gated_act_mxfp8_grad(z(4, 64), z(4, 128, dtype=U8), z(4, 4, dtype=U8), out_dtype=torch.float16), "out_dtype"),
    (lambda: B.ragged_dot_k(z(4, 64, dtype=U8), z(4, 8, dtype=BF), z(2, dtype=I32)), "lhs_scale"),
    (lambda: B.ragged_dot_k(z(4, 64, dtype=U8), z(4, 8), z(2, dtype=I32), lhs_scale=z(4, 2, dtype=U8)), "dout has dtype"),
    (lambda: B.ragged_dot_k(z(4, 64), z(4, 8), z(2, dtype=I32), lhs_scale=z(4, 2, dtype=U8)), "only with e4m3"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3)), "exactly one"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), row_group=z(4, dtype=I32)), "exactly one"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 32), z(2, 5, 3), z(2, dtype=I32)), "x has k"), (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 4), z(2, dtype=I32)), "are expected"),
    (lambda: B.ragged_lora(z(4, 64), z(3, 3, 64), z(2, 5, 3), z(2, dtype=I32)), "are expected"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3), z(3, dtype=I32)), "group_sizes has shape"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3), row_group=z(3, dtype=I32)), "row_group has shape"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), base=z(4, 6)), "base has shape"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), base=z(4, 5), out_dtype=BF), "out_dtype"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), scaling=z(2, dtype=BF)), "scaling has dtype"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), v=z(4, 4)), "v has shape"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64, dtype=BF), z(2, 5, 3), z(2, dtype=I32)), "a has dtype"),
    (lambda: B.ragged_lora(z(64, 4).t(), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32)), "unit column stride"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), workspace=z(16, dtype=U8)), "workspace holds"),
    (lambda: B.ragged_lora(z(4, 64), z(2, 300, 64), z(2, 5, 300), z(2, dtype=I32)), "workspace size"),
    (lambda: B.ragged_lora_grad(z(4, 64), z(4, 3), z(4, 6), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32)), "dout has n"),
    (lambda: B.ragged_lora_grad(z(4, 64, dtype=U8), z(4, 3), z(4, 5), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32)), "e4m3 rows go with bf16"),
    (lambda: B.ragged_lora_grad(z(4, 64, dtype=U8), z(4, 3), z(4, 5, dtype=BF), z(2, 3, 64, dtype=BF), z(2, 5, 3, dtype=BF), z(2, dtype=I32)), "need x_scale"),
    (lambda: B.ragged_lora_grad(z(4, 64), z(4, 3), z(4, 5), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), x_scale=z(4, 2, dtype=U8)), "only with e4m3"),
    (lambda: B.ragged_lora_grad(z(4, 64), z(4, 3), z(4, 5), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), dbase=z(4, 64), need_dx=False), "need_dx"),
    (lambda: B.ragged_lora_grad(z(4, 64), z(4, 4), z(4, 5), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32)), "v has shape"),
    (lambda: B.ragged_lora_grad(z(4, 64), z(4, 3), z(4, 5), z(2, 3, 64), z(2, 5, 3), z(2, dtype=I32), out=(None, z(2, 3, 64), z(2, 5, 3, dtype=BF))), "db has dtype"),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_binding_refuses(case, monkeypatch):
    device_blind(monkeypatch)
    call, text = REFUSED[case]
    with pytest.raises(ValueError, match=text):
        call()
