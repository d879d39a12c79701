"""GPU parity of moe_permute_grad and moe_unpermute_grad against the fp64 oracle.

Bounds: an fp32 sum of j terms is off by at most j 2^-24 of the sum of magnitudes, a product by 2^-24; a bf16
result adds half a step, 2^-8 of the value.  A dot product over n columns is summed by at least 64 lanes, so
no term passes through more than n / 64 + 32 additions.
"""
import numpy as np
import pytest
import torch

import oracle
from group_gemm_amd import _binding as B
from group_gemm_amd import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print("[case]", *a, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def val(t):
    return t.double().cpu().numpy()


def raw(t):
    return W.to_numpy_raw(t)


def routing(r, tokens, top_k, g, drop):
    e = r.integers(0, g, (tokens, top_k))
    e[r.random((tokens, top_k)) < drop] = -1
    _, _, _, s2c, c2s = oracle.moe_permute(np.zeros((tokens, 1), np.float32), e, g)
    return s2c, c2s


def guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), float("nan"), dtype=dtype, device=DEV)

    def check():
        assert torch.isnan(torch.cat([buf[:64], buf[64 + n:]])).all(), "wrote outside its output"
    return buf[64:64 + n].view(shape), check


SHAPES = [(1, 1, 1, 0.0), (1, 2, 8, 0.0), (3, 1, 1030, 0.3), (61, 3, 515, 0.25), (40, 8, 512, 0.1), (19, 11, 2056, 0.2),
          (7, 17, 96, 0.5), (130, 2, 7168, 0.0), (5, 4, 4104, 1.0), (257, 6, 64, 0.05)]


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_permute_grad(shape, types):
    tokens, top_k, k, drop = SHAPES[shape]
    say("permute_grad", SHAPES[shape], types)
    r = np.random.default_rng(shape)
    _, c2s = routing(r, tokens, top_k, 9, drop)
    d = dev(r.standard_normal((tokens * top_k, k)).astype(np.float32)).to(types[0])
    dx, check = guarded((tokens, k), types[1])
    B.moe_permute_grad(d, dev(c2s), top_k, out=dx)
    want = oracle.moe_permute_grad(raw(d), c2s, top_k)
    mag = oracle.moe_permute_grad(np.abs(val(d)).astype(np.float32), c2s, top_k)
    bound = top_k * 2.0 ** -24 * mag + (2.0 ** -8 * (np.abs(want) + top_k * 2.0 ** -24 * mag) if types[1] == BF else 0)
    assert (np.abs(val(dx) - want) <= bound).all()
    check()
    if types[0] == types[1]:
        assert torch.equal(B.moe_permute_grad(d, dev(c2s), top_k), dx)


def check_unpermute(dout, y, c2s, s2c, w):
    tokens, top_k = w.shape
    n = y.shape[1]
    dy, c1 = guarded(y.shape, y.dtype)
    dw, c2 = guarded((tokens, top_k), F32)
    B.moe_unpermute_grad(dout, y, dev(c2s), dev(s2c), dev(w), out=(dy, dw))
    want_y, want_w, mag = oracle.moe_unpermute_grad(raw(dout), raw(y), c2s, s2c, w)
    by = 2.0 ** -24 * np.abs(want_y) + (2.0 ** -8 * 1.001 * np.abs(want_y) if y.dtype == BF else 0)
    assert (np.abs(val(dy) - want_y) <= by).all()
    assert (np.abs(val(dw) - want_w) <= (n / 64 + 32) * 2.0 ** -24 * mag).all()
    c1(), c2()
    return dy, dw


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_unpermute_grad(shape, dtype):
    tokens, top_k, n, drop = SHAPES[shape]
    say("unpermute_grad", SHAPES[shape], dtype)
    r = np.random.default_rng(100 + shape)
    s2c, c2s = routing(r, tokens, top_k, 9, drop)
    dout, y = (dev(r.standard_normal((m, n)).astype(np.float32)).to(dtype) for m in (tokens, tokens * top_k))
    w = r.standard_normal((tokens, top_k)).astype(np.float32)
    dy, dw = check_unpermute(dout, y, c2s, s2c, w)
    a, b = B.moe_unpermute_grad(dout, y, dev(c2s), dev(s2c), dev(w))
    assert torch.equal(a, dy) and torch.equal(b, dw)
    # the same rows 2 or 4 bytes off their 16-byte alignment take the element-wise path: within the same bounds
    off = [torch.empty(t.numel() + 1, dtype=dtype, device=DEV)[1:].view(t.shape).copy_(t) for t in (dout, y)]
    check_unpermute(off[0], off[1], c2s, s2c, w)


@pytest.mark.parametrize("n", [40, 43])
def test_unpermute_grad_of_arrays_that_no_permute_wrote(n):
    """The same sorted row named twice, rows that nothing names, entries out of range: each row of dy is still
    written once, by the copy that both arrays name, and nothing is read out of bounds."""
    say("index arrays", n)
    r = np.random.default_rng(11)
    tokens, top_k = 30, 4
    M = tokens * top_k
    c2s = r.integers(0, M, M).astype(np.int32)
    c2s[r.random(M) < 0.2] = -1
    c2s[3], c2s[17], c2s[40] = M, 2 ** 31 - 1, -2 ** 31
    s2c = r.integers(-1, M, M).astype(np.int32)
    for i in range(0, M, 2):
        if 0 <= c2s[i] < M:
            s2c[c2s[i]] = i
    s2c[5], s2c[6] = M, 2 ** 31 - 1
    dout, y = (dev(r.standard_normal((m, n)).astype(np.float32)) for m in (tokens, M))
    w = r.standard_normal((tokens, top_k)).astype(np.float32)
    first = check_unpermute(dout, y, c2s, s2c, w)
    again = check_unpermute(dout, y, c2s, s2c, w)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    B.moe_permute_grad(y, dev(c2s), top_k)


def test_infinities_stay_in_their_rows():
    say("infinities")
    tokens, top_k, n = 6, 2, 24
    r = np.random.default_rng(12)
    s2c, c2s = routing(r, tokens, top_k, 3, 0.0)
    c2s[0] = -1                                        # copy 0 is not routed: its row keeps no owner
    y = r.standard_normal((tokens * top_k, n)).astype(np.float32)
    y[int(np.flatnonzero(s2c == 0)[0])] = np.nan       # the row that no copy reaches
    y[c2s[5], 3] = np.inf
    dout, w = r.standard_normal((tokens, n)).astype(np.float32), r.random((tokens, top_k)).astype(np.float32)
    dy, dw = B.moe_unpermute_grad(dev(dout), dev(y), dev(c2s), dev(s2c), dev(w))
    assert torch.isfinite(dy).all() and not dy[int(np.flatnonzero(s2c == 0)[0])].any()
    assert dw[0, 0] == 0 and torch.isinf(dw[2, 1]) and torch.isfinite(dw).sum() == tokens * top_k - 1
    dx = B.moe_permute_grad(dev(y), dev(c2s), top_k)
    assert torch.isfinite(dx).sum() == tokens * n - 1


def test_refusals():
    say("refusals")
    d = torch.zeros(12, 16, device=DEV)
    i = torch.zeros(12, dtype=torch.int32, device=DEV)
    w = torch.zeros(6, 2, device=DEV)
    for bad in (lambda: B.moe_permute_grad(d, i, 5), lambda: B.moe_permute_grad(d, i, 0), lambda: B.moe_permute_grad(d.half(), i, 2),
                lambda: B.moe_permute_grad(d, i[:6], 2), lambda: B.moe_permute_grad(d, i.long(), 2), lambda: B.moe_permute_grad(d.t(), i, 2),
                lambda: B.moe_permute_grad(d, i, 2, out=torch.zeros(5, 16, device=DEV)),
                lambda: B.moe_unpermute_grad(d[:5], d, i, i, w), lambda: B.moe_unpermute_grad(d[:6].to(BF), d, i, i, w),
                lambda: B.moe_unpermute_grad(d[:6], d, i, i, w.double()), lambda: B.moe_unpermute_grad(d[:6], d, i[:4], i, w),
                lambda: B.moe_unpermute_grad(d[:6], d, i, i, w, out=(d[:6], None)), lambda: B.moe_unpermute_grad(d[:6], d, i, i, w[:, :1])):
        with pytest.raises(ValueError):
            bad()
    assert B.moe_permute_grad(torch.zeros(0, 16, device=DEV), i[:0], 2).shape == (0, 16)
    dy, dw = B.moe_unpermute_grad(torch.zeros(3, 0, device=DEV), torch.zeros(6, 0, device=DEV), i[:6], i[:6], w[:3])
    assert dy.shape == (6, 0) and dw.tolist() == [[0, 0]] * 3


def test_backward_of_a_layer_over_mxfp4_weights():
    """out = un-permute(product(permute(x))) with frozen 4-bit weights: the gradients of x and of the router
    weights by moe_unpermute_grad, ragged_dot_m over the dequantised weights and moe_permute_grad, against the
    same chain in 64 bits and against differences of the 64-bit forward; then captured and replayed."""
    say("backward of a layer")
    tokens, top_k, g, k, n = 24, 2, 5, 64, 48
    r = np.random.default_rng(13)
    wq, wsc = B.mxfp4_quantize_weights(dev(r.standard_normal((g, k, n)) / np.sqrt(k)).to(BF))
    wv = oracle.mxfp4_values(wq.view(torch.uint8).cpu().numpy(), wsc.cpu().numpy())     # [g, n, k]
    x = dev(r.standard_normal((tokens, k)).astype(np.float32))
    experts = dev(r.integers(0, g, (tokens, top_k)).astype(np.int32))
    rw = dev(r.random((tokens, top_k)).astype(np.float32))
    dout = dev(r.standard_normal((tokens, n)).astype(np.float32))
    wd = B.mxfp4_dequantize(wq, wsc, out_dtype=F32)

    def backward():
        sx, _, gs, s2c, c2s = B.moe_permute(x, experts, g)
        y = B.ragged_dot_m(sx, wd.transpose(1, 2).contiguous(), gs)
        dy, dw = B.moe_unpermute_grad(dout, y, c2s, s2c, rw)
        return B.moe_permute_grad(B.ragged_dot_m(dy, wd, gs), c2s, top_k), dw

    dx, dw = backward()

    def forward64(xv, wv_):
        e = experts.cpu().numpy()
        out = np.zeros((tokens, n))
        for t in range(tokens):
            for j in range(top_k):
                out[t] += wv_[t, j] * (wv[e[t, j]] @ xv[t])
        return out

    xv, rv, dv = val(x), val(rw), val(dout)
    e = experts.cpu().numpy()
    want_x = np.stack([sum(rv[t, j] * (dv[t] @ wv[e[t, j]]) for j in range(top_k)) for t in range(tokens)])
    want_w = np.array([[dv[t] @ (wv[e[t, j]] @ xv[t]) for j in range(top_k)] for t in range(tokens)])
    mag_x = np.stack([sum(rv[t, j] * (np.abs(dv[t]) @ np.abs(wv[e[t, j]])) for j in range(top_k)) for t in range(tokens)])
    mag_w = np.array([[np.abs(dv[t]) @ (np.abs(wv[e[t, j]]) @ np.abs(xv[t])) for j in range(top_k)] for t in range(tokens)])
    # fp32 throughout: the roundings of the two chained sums, each term in fewer than n + k + 8 of them
    assert (np.abs(val(dx) - want_x) <= (n + k + 8) * 2.0 ** -23 * mag_x).all()
    assert (np.abs(val(dw) - want_w) <= (n + k + 8) * 2.0 ** -23 * mag_w).all()
    h = 2.0 ** -10   # the loss is linear in each: central differences are exact but for 64-bit rounding
    for t, c in ((0, 0), (7, 33), (23, 63)):
        d = np.zeros_like(xv)
        d[t, c] = h
        diff = ((forward64(xv + d, rv) - forward64(xv - d, rv)) * dv).sum() / (2 * h)
        assert abs(float(dx[t, c]) - diff) <= (n + k + 8) * 2.0 ** -23 * mag_x[t, c] + 1e-9
    for t, j in ((0, 0), (11, 1), (23, 1)):
        d = np.zeros_like(rv)
        d[t, j] = h
        diff = ((forward64(xv, rv + d) - forward64(xv, rv - d)) * dv).sum() / (2 * h)
        assert abs(float(dw[t, j]) - diff) <= (n + k + 8) * 2.0 ** -23 * mag_w[t, j] + 1e-9

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            cx, cw = backward()
    for seed in range(3):
        q = np.random.default_rng(50 + seed)
        x.copy_(dev(q.standard_normal((tokens, k)).astype(np.float32)))
        experts.copy_(dev(q.integers(-1, g, (tokens, top_k)).astype(np.int32)))
        dout.copy_(dev(q.standard_normal((tokens, n)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        ex, ew = backward()
        assert torch.equal(cx, ex) and torch.equal(cw, ew), seed


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 15, 511, 512, 513, 521, 1031])
@pytest.mark.parametrize("top_k", [1, 2, 3, 5, 9])
def test_widths_of_any_alignment(n, top_k, dtype):
    """Rows that begin at any element, a last piece that overlaps the one before, every batch of copies: the
    un-permute and both gradients, with every output behind an odd element."""
    say("widths", n, top_k, dtype)
    tokens = 37
    r = np.random.default_rng(n + top_k)
    s2c, c2s = routing(r, tokens, top_k, 5, 0.2)
    c2s_d, s2c_d = dev(c2s), dev(s2c)
    M = tokens * top_k

    def odd(shape):
        b = torch.full((int(np.prod(shape)) + 66,), float("nan"), dtype=dtype, device=DEV)
        return b[33:33 + int(np.prod(shape))].view(shape), lambda: torch.isnan(torch.cat([b[:33], b[-33:]])).all()

    y, _ = odd((M, n))
    y.copy_(dev(r.standard_normal((M, n)).astype(np.float32)))
    dout, _ = odd((tokens, n))
    dout.copy_(dev(r.standard_normal((tokens, n)).astype(np.float32)))
    w = dev(r.standard_normal((tokens, top_k)).astype(np.float32))
    routed = (c2s >= 0)[:, None]
    rows = np.where(routed, val(y)[np.maximum(c2s, 0)], 0.0).reshape(tokens, top_k, n)
    step = 2.0 ** -8 if dtype == BF else 0.0

    for weights, call in ((val(w), lambda o: B.moe_unpermute(y, c2s_d, w, out=o)), (np.ones((tokens, top_k)), lambda o: B.moe_permute_grad(y, c2s_d, top_k, out=o))):
        out, ok = odd((tokens, n))
        call(out)
        want, mag = (rows * weights[..., None]).sum(1), (np.abs(rows * weights[..., None])).sum(1)
        # top_k products and additions, each rounded once to fp32, and the result's own rounding
        bound = (top_k + 1) * 2.0 ** -23 * mag
        assert (np.abs(val(out) - want) <= bound + step * (np.abs(want) + bound)).all() and ok()

    dy, ok = odd((M, n))
    dw = torch.empty(tokens, top_k, device=DEV)
    B.moe_unpermute_grad(dout, y, c2s_d, s2c_d, w, out=(dy, dw))
    want = np.zeros((M, n))
    at = np.nonzero(c2s >= 0)[0]
    want[c2s[at]] = val(w).reshape(-1)[at, None] * val(dout)[at // top_k]
    assert (np.abs(val(dy) - want) <= (2.0 ** -24 + step * 1.01) * np.abs(want)).all() and ok()
    terms = rows * val(dout)[:, None]
    assert (np.abs(val(dw) - terms.sum(-1)) <= (n / 64 + 34) * 2.0 ** -24 * np.abs(terms).sum(-1)).all()


def test_gradients_past_32_bits():
    """More than 2^32 elements: a few tokens far apart, their copies in the last rows."""
    say("large rows")
    tokens, top_k, n = 41003, 2, 57345
    M = tokens * top_k
    assert M * n > 2 ** 32
    c2s = torch.arange(M - 1, -1, -1, dtype=torch.int32, device=DEV)   # copy i in row M - 1 - i
    s2c = c2s.clone()
    y = torch.zeros(M, n, dtype=BF, device=DEV)
    some = torch.tensor([0, 1, tokens // 2, tokens - 2, tokens - 1], device=DEV)
    for t in some.tolist():
        y[M - 2 - 2 * t:M - 2 * t] = torch.randn(2, n, device=DEV).to(BF)
    dout = torch.zeros(tokens, n, dtype=BF, device=DEV)
    dout[some] = torch.randn(5, n, device=DEV).to(BF)
    w = torch.rand(tokens, top_k, device=DEV)
    dx = B.moe_permute_grad(y, c2s, top_k)
    dy, dw = B.moe_unpermute_grad(dout, y, c2s, s2c, w)
    for t in some.tolist():
        a, b = y[M - 1 - 2 * t], y[M - 2 - 2 * t]   # copies 2 t and 2 t + 1
        assert torch.equal(dx[t], (a.float() + b.float()).to(BF))
        for j, row in ((0, M - 1 - 2 * t), (1, M - 2 - 2 * t)):
            assert torch.equal(dy[row], (w[t, j] * dout[t].float()).to(BF))
            p = dout[t].double() * y[row].double()
            assert abs(dw[t, j].double() - p.sum()) <= (n / 64 + 34) * 2.0 ** -24 * p.abs().sum()
    assert not dx[3].any() and not dy[5].any() and not dy[M - 9].any()


def test_gradients_in_place_are_refused():
    say("in place")
    b = torch.zeros(20, 16, device=DEV)
    y, dout, i, w = b[:12], torch.zeros(6, 16, device=DEV), torch.arange(12, dtype=torch.int32, device=DEV), torch.ones(6, 2, device=DEV)
    for dy in (y, b[8:20]):
        with pytest.raises(ValueError):
            B.moe_unpermute_grad(dout, y, i, i, w, out=(dy, None))
    B.moe_unpermute_grad(dout, y, i, i, w, out=(torch.empty_like(y), None))


def test_no_tokens():
    say("no tokens")
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert B.moe_permute_grad(torch.zeros(0, 24, device=DEV), i, 3).shape == (0, 24)
    dy, dw = B.moe_unpermute_grad(torch.zeros(0, 24, device=DEV), torch.zeros(0, 24, device=DEV), i, i, torch.zeros(0, 3, device=DEV))
    assert dy.shape == (0, 24) and dw.shape == (0, 3)
