"""Pins of the MXFP4 and MoE-gradient oracles (CPU): the format by hand and against torch's fp32
arithmetic, the gradients against differences of the forward oracles."""
import numpy as np
import pytest

import oracle


def test_e2m1_values_and_packing():
    codes = np.array([[0x10 * (2 * i + 1) + 2 * i for i in range(8)] + [0] * 8], dtype=np.uint8)   # codes 0 .. 15, zeros
    v = oracle.mxfp4_values(codes, oracle.mxfp4_panels(np.array([[128]])))
    assert v[0, :16].tolist() == [0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12]
    assert np.isnan(oracle.mxfp4_values(codes, oracle.mxfp4_panels(np.array([[255]])))).all()
    assert oracle.mxfp4_values(codes, oracle.mxfp4_panels(np.array([[0]])))[0, 1] == 2.0 ** -128


@pytest.mark.parametrize("kb", [1, 7, 8, 9, 17])
def test_panels(kb):
    s = np.arange(1, 3 * kb + 1, dtype=np.uint8).reshape(3, kb)
    p = oracle.mxfp4_panels(s)
    assert p.shape == (-(-kb // 8), 3, 8)
    for r in range(3):
        for b in range(8 * p.shape[0]):
            assert p[b // 8, r, b % 8] == (s[r, b] if b < kb else 0)


def test_quantize_ties_saturation_and_specials():
    x = np.zeros((1, 32))
    x[0, :12] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 7.9, -7.9, -0.0]   # max 7.9: E = 0
    codes, s = oracle.mxfp4_quantize(x)
    assert s.tolist() == [[127]]
    v = oracle.mxfp4_values(codes, oracle.mxfp4_panels(s))[0]
    assert v[:12].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, -4, 6, -6, 0] and np.signbit(v[11])
    assert oracle.mxfp4_quantize(np.zeros((1, 32)))[1].tolist() == [[0]]
    assert oracle.mxfp4_quantize(np.full((1, 32), 2.0 ** -140))[1].tolist() == [[0]]
    for bad in (np.inf, -np.inf, np.nan):
        y = x.copy()
        y[0, 20] = bad
        assert oracle.mxfp4_quantize(y)[1].tolist() == [[255]]


def test_quantize_is_nearest():
    r = np.random.default_rng(5)
    x = r.standard_normal((7, 96)) * 2.0 ** r.integers(-30, 30, (7, 1))
    codes, s = oracle.mxfp4_quantize(x)
    v = oracle.mxfp4_values(codes, oracle.mxfp4_panels(s))
    scale = np.repeat(2.0 ** (s.astype(float) - 127), 32, axis=1)
    grid = np.concatenate([oracle.E2M1, -oracle.E2M1])
    best = np.abs(x[..., None] - grid * scale[..., None]).min(-1)
    assert np.array_equal(np.abs(x - v), best)
    assert (np.abs(x).reshape(7, 3, 32).max(-1) / 2.0 ** (s.astype(float) - 127) < 8).all()


def test_product_is_the_sum_over_k():
    r = np.random.default_rng(6)
    m, k, n, gs = 9, 64, 5, [2, 0, 4, -3, 1]
    lc, ls = oracle.mxfp4_quantize(r.standard_normal((m, k)))
    rc, rs = oracle.mxfp4_quantize(r.standard_normal((5, n, k)))
    lp, rp = oracle.mxfp4_panels(ls), oracle.mxfp4_panels(rs)
    out, mag = oracle.ragged_dot_m_mxfp4(lc, lp, rc, rp, gs)
    a, b = oracle.mxfp4_values(lc, lp), oracle.mxfp4_values(rc, rp)
    for row, h in zip(range(m), [0, 0, 2, 2, 2, 2, 4]):
        for col in range(n):
            assert out[row, col] == pytest.approx(sum(a[row, i] * b[h, col, i] for i in range(k)), rel=1e-12, abs=1e-12)
            assert mag[row, col] >= abs(out[row, col]) - 1e-12
    assert not out[7:].any()


def _routing(r, tokens, top_k, g):
    experts = r.integers(-1, g, (tokens, top_k))   # -1: not routed
    return oracle.moe_permute(np.zeros((tokens, 1), np.float32), experts, g)


def test_gradients_against_differences():
    r = np.random.default_rng(7)
    tokens, top_k, g, k = 5, 3, 4, 6
    _, _, _, s2c, c2s = _routing(r, tokens, top_k, g)
    M = tokens * top_k
    x = r.standard_normal((tokens, k))
    ds = r.standard_normal((M, k))

    def permuted(x):
        out = np.zeros((M, k))
        for p, i in enumerate(s2c):
            if i >= 0:
                out[p] = x[i // top_k]
        return out

    # forward by the oracle itself (fp32 rows, whole numbers, so nothing is rounded)
    xi = r.integers(-8, 9, (tokens, k)).astype(np.float32)
    e = np.full(M, -1)
    e[c2s >= 0] = 0
    assert np.array_equal(np.sort(permuted(xi), axis=0), np.sort(oracle.moe_permute(xi, e.reshape(tokens, top_k), 1)[0], axis=0))
    dx = oracle.moe_permute_grad(ds.astype(np.float32), c2s, top_k)
    ds32 = ds.astype(np.float32).astype(np.float64)
    for t in range(tokens):
        for c in range(k):
            d = np.zeros_like(x)
            d[t, c] = 1e-3
            diff = ((permuted(x + d) - permuted(x - d)) * ds32).sum() / 2e-3
            assert dx[t, c] == pytest.approx(diff, abs=1e-9)

    y, w, dout = (r.standard_normal(s).astype(np.float32) for s in ((M, k), (tokens, top_k), (tokens, k)))
    dy, dw, _ = oracle.moe_unpermute_grad(dout, y, c2s, s2c, w)

    def loss(y, w):
        return float((oracle.moe_unpermute(y, c2s, w) * dout).sum())

    h = 2.0 ** -6   # the loss is linear in y and in w: a central difference is exact but for rounding
    for p in range(M):
        for c in range(k):
            d = np.zeros_like(y, dtype=np.float64)
            d[p, c] = h
            assert dy[p, c] == pytest.approx((loss(y + d, w) - loss(y - d, w)) / (2 * h), abs=1e-9)
    for t in range(tokens):
        for j in range(top_k):
            d = np.zeros_like(w, dtype=np.float64)
            d[t, j] = h
            assert dw[t, j] == pytest.approx((loss(y, w + d) - loss(y, w - d)) / (2 * h), abs=1e-9)
