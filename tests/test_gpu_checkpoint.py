"""GPU tests of the 8-bit activation checkpoints against the fp64 oracle: MXFP8 rows and back, the gated unit and its
backward pass, and the weight gradient from rows kept in 8 bits.

Bounds.  Codes, scales and values are exact.  The gated unit in fp32: y (the gate, or 2 sqrt(2/pi) (x + c x^3)) is off by
4 roundings, e^-y by 2 ulp and that error of y, the rest by a rounding an operation, so a value of size F is off by
(4 |y| + 16) 2^-24 F, its slope by twice that of the sum of its terms' magnitudes; past |y| = 88 p is held, which is
1e-36 of the operands.  A sum of `rows` products is off by (rows + 40) 2^-24 of the sum of magnitudes.  A result adds
half a step of its type: 2^-8 (bf16) or 2^-24 of its value.
"""
import numpy as np
import pytest
import torch

import group_gemm_amd as G
import oracle
from group_gemm_amd import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E = 2.0 ** -24


def say(*a):
    print("[case]", *a, flush=True)


def val(t):
    return t.double().cpu().numpy()


def half(t):
    return {BF: 2.0 ** -8, F32: E}[t]


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def rows(seed, m, k, dtype):
    r = np.random.default_rng(seed)
    x = r.standard_normal((m, k)) * np.exp(0.5 * r.standard_normal(k))
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(DEV)


def framed(shape, dtype, fill=None):
    """A tensor between two strips that have to stay as they are."""
    n = int(np.prod(shape))
    size = torch.empty((), dtype=dtype).element_size()
    buf = torch.full(((n + 128) * size,), 0xA5, dtype=torch.uint8, device=DEV)
    t = buf[64 * size:(64 + n) * size].view(dtype).view(shape)

    def check():
        rest = torch.cat([buf[:64 * size], buf[(64 + n) * size:]])
        assert bool((rest == 0xA5).all()), "wrote outside its output"
    return t, check


SHAPES = [(1, 32), (1, 4096), (3, 96), (27, 2880), (61, 1056), (257, 64), (40, 7168), (1025, 32)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_there_and_back(shape, dtype):
    say("rows", shape, dtype)
    x = rows(sum(shape), *shape, dtype)
    codes, c1 = framed(shape, E4M3)
    scale, c2 = framed((shape[0], shape[1] // 32), torch.uint8)
    G.mxfp8_quantize(x, out=(codes, scale))
    want_c, want_s = oracle.mxfp8_quantize(val(x))
    c1(), c2()
    assert np.array_equal(u8(codes), want_c) and np.array_equal(u8(scale), want_s)
    want = oracle.mxfp8_values(want_c, want_s)
    for out_dtype in (BF, F32):
        out, c3 = framed(shape, out_dtype)
        G.mxfp8_dequantize(codes, scale, out=out)
        c3()
        assert np.array_equal(val(out), want)
    assert (np.abs(want - val(x)) <= 2.0 ** -4 * np.abs(val(x)) + np.repeat(2.0 ** (want_s.astype(float) - 137), 32, 1)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_with_a_stride_and_any_alignment(dtype):
    say("strided rows", dtype)
    wide = rows(7, 33, 1 + 416 + 3, dtype)
    x = wide[:, 1:417]
    codes, scale = G.mxfp8_quantize(x)
    want_c, want_s = oracle.mxfp8_quantize(val(x))
    assert np.array_equal(u8(codes), want_c) and np.array_equal(u8(scale), want_s)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_whole_range_of_values(dtype):
    say("range", dtype)
    r = np.random.default_rng(5)
    exps = np.arange(-149 if dtype == F32 else -133, 128)
    x = np.ldexp(1 + r.integers(0, 128, (len(exps), 64)) / 128.0, exps[:, None]) * r.choice([-1, 1], (len(exps), 64))
    x[:, 33:] = np.ldexp(x[:, 33:], -r.integers(0, 20, (len(exps), 31)))
    x[0, :32] = 0
    x[5, 0] = -0.0
    # fractions next to the scale's border and on the grid's midpoints
    x[40, :4] = np.ldexp([1.75, 1.0, 1.0625, 1.1875], exps[40])
    x[41, :4] = np.ldexp([1.7578125, 1.0, 1.0625, -1.1875], exps[41])
    t = torch.from_numpy(x.astype(np.float32)).to(dtype).to(DEV)
    codes, scale = G.mxfp8_quantize(t)
    want_c, want_s = oracle.mxfp8_quantize(val(t))
    assert np.array_equal(u8(scale), want_s)
    assert np.array_equal(u8(codes), want_c)
    back = oracle.mxfp8_values(want_c, want_s)
    back = np.where(np.abs(back) >= 2.0 ** 128, np.copysign(np.inf, back), back)   # rounded up past the largest number
    normal = np.abs(back) >= 2.0 ** -126
    got = val(G.mxfp8_dequantize(codes, scale, out_dtype=F32))
    assert np.array_equal(got[normal], back[normal]) and (np.abs(got[~normal] - back[~normal]) <= 2.0 ** -126).all()


def test_infinities_and_nan_stay_in_their_blocks():
    say("non-finite blocks")
    x = rows(9, 4, 128, BF)
    x[0, 5], x[1, 40], x[2, 127] = float("inf"), float("-inf"), float("nan")
    codes, scale = G.mxfp8_quantize(x)
    bad = np.zeros((4, 4), bool)
    bad[0, 0] = bad[1, 1] = bad[2, 3] = True
    assert np.array_equal(u8(scale) == 255, bad)
    for t in (BF, F32):
        assert np.array_equal(np.isnan(val(G.mxfp8_dequantize(codes, scale, out_dtype=t))), np.repeat(bad, 32, 1))
    h, codes, scale = G.gated_act_mxfp8(x, torch.ones_like(x))
    assert np.array_equal(np.isfinite(val(h)), np.isfinite(val(x)))
    dg, du, h = G.gated_act_mxfp8_grad(torch.ones_like(x), codes, scale)
    for t in (dg, du, h):
        assert np.array_equal(np.isnan(val(t)), np.repeat(bad, 32, 1))


def test_every_code_and_scale_byte():
    say("all codes")
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1)
    scale = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None].repeat(1, 8).contiguous()
    want = oracle.mxfp8_values(u8(codes), u8(scale))
    for t in (BF, F32):
        got = val(G.mxfp8_dequantize(codes, scale, out_dtype=t))
        with np.errstate(over="ignore"):
            ok = np.abs(want) < 2.0 ** 128
        big = np.abs(want) >= 2.0 ** 128
        normal = np.abs(want) >= 2.0 ** -126
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[ok & normal], want[ok & normal]) and np.isinf(got[big]).all()
        assert (np.abs(got[ok & ~normal] - want[ok & ~normal]) <= 2.0 ** -126).all()


# ---------------------------------------------------------------------------------------------------------------
# the gated unit


def gate_bounds(g, act):
    """|act| and the slope's terms, each with its error."""
    x = np.abs(g)
    y = x if act == "silu" else 1.6 * (x + 0.0448 * x ** 3)
    slope_y = 1.0 if act == "silu" else 1.6 * (1 + 0.135 * x * x)
    rel = (4 * np.minimum(y, 90) + 16) * E
    f, _ = oracle.gate_and_slope(g, act)
    p = np.abs(f) / np.maximum(x, 1e-30)
    p = np.where(x < 1e-30, 0.5, p)
    terms = p + np.minimum(x * p * np.minimum(1 - p + 1e-30, 1) * slope_y, 1e3)
    return rel * np.abs(f) + 1e-36 * x, 2 * rel * terms + 1e-36 * (1 + x)


def within(got, want, bound, what=""):
    off = ~(np.abs(got - want) <= bound)
    i = tuple(np.argwhere(off)[0]) if off.any() else None
    assert i is None, f"{what}: {int(off.sum())} of {off.size} off, first {i}: {got[i]!r}, not {want[i]!r}, bound {bound[i]!r}"


def check_h(h, g, u, act):
    f, _ = oracle.gate_and_slope(g, act)
    ef, _ = gate_bounds(g, act)
    want = f * u
    within(val(h), want, ef * np.abs(u) + (half(h.dtype) + E) * np.abs(want) * 1.01 + 1e-38, "h")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("shape", [(1, 32), (27, 2880), (61, 1056), (257, 64), (5, 14336)])
def test_gated(shape, types, act):
    say("gated", shape, types, act)
    g, u = rows(1, *shape, types[0]), rows(2, *shape, types[0])
    m, n = shape
    h, c0 = framed(shape, types[1])
    codes, c1 = framed((m, 2 * n), E4M3)
    scale, c2 = framed((m, n // 16), torch.uint8)
    G.gated_act_mxfp8(g, u, act=act, out=(h, codes, scale))
    c0(), c1(), c2()
    want_c, want_s = oracle.mxfp8_quantize(np.concatenate([val(g), val(u)], 1))
    assert np.array_equal(u8(codes), want_c) and np.array_equal(u8(scale), want_s)
    check_h(h, val(g), val(u), act)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("shape", [(1, 32), (27, 2880), (61, 1056), (257, 64), (5, 14336)])
def test_gated_grad(shape, types, act):
    say("gated_grad", shape, types, act)
    m, n = shape
    codes, scale = G.mxfp8_quantize(rows(3, m, 2 * n, F32))
    dh = rows(4, m, n, types[0])
    out = [framed(shape, types[1]) for _ in range(3)]
    G.gated_act_mxfp8_grad(dh, codes, scale, act=act, out=tuple(t for t, _ in out))
    for _, c in out:
        c()
    x = oracle.mxfp8_values(u8(codes), u8(scale))
    g, u, d = x[:, :n], x[:, n:], val(dh)
    want = oracle.gated_act_grad(d, g, u, act)
    ef, es = gate_bounds(g, act)
    r = (half(types[1]) + 2 * E) * 1.01
    for (got, _), w, e in zip(out, want, (np.abs(d * u) * es, np.abs(d) * ef, np.abs(u) * ef)):
        within(val(got), w, e + r * np.abs(w) + 1e-38)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_at_large_gates(act):
    """Gates past the exponential's range: finite, and the unit's limits."""
    g = torch.tensor([0.0, -0.0, 1e-30, 20, -20, 87, -87, 89, -89, 100, -100, 1e4, -1e4, 3e38, -3e38, 1e19], device=DEV).repeat(2)[None].contiguous()
    u = torch.full_like(g, 0.5)
    h, codes, scale = G.gated_act_mxfp8(g, u, act=act)
    want, _ = oracle.gate_and_slope(np.clip(val(g), -1e5, 1e5), act)
    want = np.where(np.abs(val(g)) > 1e5, np.maximum(val(g), 0), want)
    assert np.isfinite(val(h)).all() and (np.abs(val(h) - 0.5 * want) <= 400 * E * np.abs(want) + 1e-35).all()
    v = torch.tensor([0.0, 20, -20, 88, -88, 96, -96, 448], device=DEV).repeat(4)[None].contiguous()
    codes, scale = G.mxfp8_quantize(torch.cat([v, torch.ones_like(v)], 1))
    dg, du, _ = G.gated_act_mxfp8_grad(torch.ones_like(v), codes, scale, act=act)
    f, d = oracle.gate_and_slope(oracle.mxfp8_values(u8(codes), u8(scale))[:, :32], act)
    assert (np.abs(val(dg) - d) <= 1e-6 * np.abs(d) + 1e-30).all() and (np.abs(val(du) - f) <= 4e-5 * np.abs(f) + 1e-35).all()


def test_halves_of_one_matrix_and_gradients_in_place():
    say("halves")
    m, n = 37, 160
    x = rows(11, m, 2 * n, BF)
    h, codes, scale = G.gated_act_mxfp8(x[:, :n], x[:, n:])
    h2, codes2, scale2 = G.gated_act_mxfp8(x[:, :n].contiguous(), x[:, n:].contiguous())
    assert torch.equal(h, h2) and torch.equal(codes.view(torch.uint8), codes2.view(torch.uint8)) and torch.equal(scale, scale2)
    dh = rows(12, m, n, BF)
    want = G.gated_act_mxfp8_grad(dh, codes, scale)
    both = torch.empty(m, 2 * n, dtype=BF, device=DEV)
    G.gated_act_mxfp8_grad(dh, codes, scale, out=(both[:, :n], both[:, n:], None))
    assert torch.equal(both, torch.cat(want[:2], 1))
    for place in range(3):
        d = dh.clone()
        got = G.gated_act_mxfp8_grad(d, codes, scale, out=tuple(d if i == place else None for i in range(3)))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------------------------------------------
# the weight gradient


def wgrad_case(seed, m, k, n, g):
    codes, scale = G.mxfp8_quantize(rows(seed, m, k, F32))
    dout = rows(seed + 1, m, n, BF)
    return codes, scale, dout, oracle.mxfp8_values(u8(codes), u8(scale)), val(dout)


def check_wgrad(out, x, d, sizes, alpha=1.0, beta=0.0, old=None):
    at, m = 0, x.shape[0]
    got, dtype = out if isinstance(out, tuple) else (val(out), out.dtype)
    for h, s in enumerate(sizes):
        s = min(max(int(s), 0), m - at)
        a, b = x[at:at + s], d[at:at + s]
        at += s
        before = beta * old[h] if beta else 0.0
        want = alpha * (a.T @ b) + before
        mag = abs(alpha) * (np.abs(a).T @ np.abs(b)) + np.abs(before)
        within(got[h], want, (s + 40) * E * mag + half(dtype) * 1.01 * np.abs(want), f"group {h}")


# rows of one, tile borders, groups without rows, rows past the last group, n without any alignment, one long group
WGRAD = [(1, 32, 1, [1]), (5, 64, 8, [0, 5, 0]), (130, 288, 264, [64, 65, 1]), (200, 160, 77, [30, 0, 100, 33]), (387, 512, 513, [1, 2, 0, 380]),
         (300, 1056, 40, [300]), (64, 96, 1447, [32, 32]), (33, 256, 256, [40, 9]), (70, 32, 250, [-4, 70]), (0, 64, 16, [0, 0]), (1100, 320, 328, [1000, 0, 100])]


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(WGRAD)))
def test_weight_gradient(case, out_dtype):
    m, k, n, sizes = WGRAD[case]
    say("wgrad", WGRAD[case], out_dtype)
    codes, scale, dout, x, d = wgrad_case(case, m, k, n, len(sizes))
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    out, c = framed((len(sizes), k, n), out_dtype)
    ws = torch.empty(G.workspace_bytes("ragged_k", m, k, n, len(sizes), 0, torch.uint8), dtype=torch.uint8, device=DEV)
    G.ragged_dot_k(codes, dout, gs, out=out, lhs_scale=scale, workspace=ws)
    c()
    check_wgrad(out, x, d, sizes)
    want = (1 if min(sizes) < 0 else 0) | (2 if sum(max(s, 0) for s in sizes) > m else 0)
    assert G.read_device_status(ws) == want


# whole 128 columns of k and whole 16 bytes of n: every count of 32-row slices up to the ring's wrap, long groups, tiles that
# end inside a wave's part, several tiles a group
RING = [(1, 128, 8, [1]), (300, 128, 264, [31, 32, 33, 64, 65, 75]), (500, 256, 256, [97, 128, 129, 146]), (700, 384, 520, [160, 161, 0, 379]),
        (1500, 640, 72, [700, 0, 333, 400]), (900, 128, 1032, [225, 256, 257, 162]), (2100, 896, 312, [2100]), (64, 1152, 2064, [40, 24]),
        (1700, 96, 40, [1500, 0, 190]), (3000, 64, 77, [2999, 1]), (900, 32, 520, [33, 867])]   # rows in parts


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(RING)))
def test_weight_gradient_in_the_ring(case, out_dtype):
    m, k, n, sizes = RING[case]
    say("wgrad ring", RING[case], out_dtype)
    codes, scale, dout, x, d = wgrad_case(20 + case, m, k, n, len(sizes))
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    out, c = framed((len(sizes), k, n), out_dtype)
    for alpha in (1.0, -0.5):
        G.ragged_dot_k(codes, dout, gs, out=out, lhs_scale=scale, alpha=alpha)
        c()
        check_wgrad(out, x, d, sizes, alpha)


def test_weight_gradient_past_32_bits():
    """dout of more than 2 GiB: the last rows of a long group, and a short one behind it."""
    say("wgrad long")
    m, k, n = 66000, 128, 16392
    codes, scale, dout = torch.zeros(m, k, dtype=torch.uint8, device=DEV), torch.zeros(m, 4, dtype=torch.uint8, device=DEV), torch.ones(m, n, dtype=BF, device=DEV)
    c, s, _, x, _ = wgrad_case(70, 40, k, 8, 1)
    codes[-40:], scale[-40:] = c.view(torch.uint8), s
    sizes = [m - 10, 7]
    out = G.ragged_dot_k(codes, dout, torch.tensor(sizes, dtype=torch.int32, device=DEV), lhs_scale=scale)
    ones = np.ones((40, 16))
    check_wgrad((val(out[:, :, -16:]), F32), x, ones, [30, 7])
    check_wgrad((val(out[:, :, :16]), F32), x, ones, [30, 7])


@pytest.mark.parametrize("m,k,n", [(150, 256, 264), (150, 288, 264), (150, 288, 263), (1700, 96, 40), (1700, 96, 41)])
@pytest.mark.parametrize("out_dtype", [F32, BF])
def test_weight_gradient_accumulates(m, k, n, out_dtype):
    say("wgrad in place", m, k, n, out_dtype)
    sizes = [m - 80, 0, 80]
    codes, scale, dout, x, d = wgrad_case(50, m, k, n, 3)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    old = torch.randn(3, k, n, device=DEV).to(out_dtype)
    out = old.clone()
    G.ragged_dot_k(codes, dout, gs, out=out, lhs_scale=scale, alpha=0.75, beta=-0.5)
    check_wgrad(out, x, d, sizes, 0.75, -0.5, val(old))


@pytest.mark.parametrize("k", [256, 288])
def test_weight_gradient_of_values_behind_the_groups(k):
    """Rows past the last group and other groups' rows hold NaN: none reaches a gradient."""
    say("wgrad NaN", k)
    m, n, sizes = 140, 264, [50, 0, 40]
    codes, scale, dout, x, d = wgrad_case(60, m, k, n, 3)
    scale[90:] = 255
    dout[90:] = float("nan")
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    check_wgrad(G.ragged_dot_k(codes, dout, gs, lhs_scale=scale), x, d, sizes)
    scale[3, 2] = 255                                    # a checkpoint's NaN block reaches its group's 32 rows alone
    got = val(G.ragged_dot_k(codes, dout, gs, lhs_scale=scale))
    bad = np.zeros((3, k), bool)
    bad[0, 64:96] = True
    assert np.array_equal(np.isnan(got).all(-1), bad) and np.array_equal(np.isnan(got).any(-1), bad)


@pytest.mark.parametrize("m,k,n", [(150, 96, 41), (150, 288, 264), (1700, 96, 40), (1700, 96, 41)])
def test_weight_gradient_of_non_finite_neighbours(m, k, n):
    """A group of NaN between two others, and NaN behind the last, reach neither, with the rows in parts too."""
    say("wgrad neighbours", m, k, n)
    sizes = [m // 2 - 3, m // 4 + 1, m // 8 + 5]
    codes, scale, dout, x, d = wgrad_case(70, m, k, n, 3)
    at = [slice(sizes[0], sum(sizes[:2])), slice(sum(sizes), m)]
    for i in at:
        scale[i], dout[i] = 255, float("inf")
    out = val(G.ragged_dot_k(codes, dout, torch.tensor(sizes, dtype=torch.int32, device=DEV), lhs_scale=scale))
    assert np.isnan(out[1]).all()
    x, d = x.copy(), d.copy()
    for i in at:
        x[i], d[i] = 0, 0
    out[1] = 0
    check_wgrad((out, F32), x, d, sizes)


# ---------------------------------------------------------------------------------------------------------------
# together, captured, on other streams


def test_layer_backward_from_checkpoints_against_differences():
    """An expert layer's up half, y = (act(x w0) * x w1) with x, gate and up kept in 8 bits.  With x, gate and up that
    8 bits hold exactly the gradients are those of the loss itself: checked against central differences in fp64."""
    say("layer")
    m, k, n, sizes = 96, 64, 64, [40, 0, 56]
    r = np.random.default_rng(3)
    x = torch.from_numpy(r.integers(-8, 9, (m, k)) / 8.0).float().to(BF).to(DEV)
    gate, up = (torch.from_numpy(r.integers(-15, 16, (m, n)) / 8.0).float().to(BF).to(DEV) for _ in range(2))
    dh = torch.from_numpy(r.standard_normal((m, n))).float().to(DEV)
    xc, xs = G.mxfp8_quantize(x)
    h, codes, scale = G.gated_act_mxfp8(gate, up, out_dtype=F32)
    assert torch.equal(G.mxfp8_dequantize(xc, xs), x) and torch.equal(G.mxfp8_dequantize(codes, scale), torch.cat([gate, up], 1))
    dg, du, h2 = G.gated_act_mxfp8_grad(dh, codes, scale)
    assert torch.equal(h, h2)
    loss = lambda a, b: (val(dh) * oracle.gate_and_slope(a, "silu")[0] * b).sum(0)
    step = 1e-4
    for i in (0, 41, 95):
        e = np.zeros((m, 1)); e[i] = step
        q = (loss(val(gate) + e, val(up)) - loss(val(gate) - e, val(up))) / (2 * step)
        assert np.abs(q - val(dg)[i]).max() < 1e-5
        q = (loss(val(gate), val(up) + e) - loss(val(gate), val(up) - e)) / (2 * step)
        assert np.abs(q - val(du)[i]).max() < 1e-5
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    dgb = dg.to(BF)
    dw = G.ragged_dot_k(xc, dgb, gs, lhs_scale=xs)
    check_wgrad(dw, val(x), val(dgb), sizes)
    assert torch.equal(dw, G.ragged_dot_k(xc, dgb, gs, lhs_scale=xs))


def test_captured_and_replayed():
    say("graph")
    m, k, n = 100, 96, 64
    gs = torch.tensor([60, 40], dtype=torch.int32, device=DEV)
    x, gu, dh = rows(1, m, k, BF), rows(2, m, 2 * n, BF), rows(3, m, n, BF)

    def step():
        xc, xs = G.mxfp8_quantize(x)
        h, c, s = G.gated_act_mxfp8(gu[:, :n], gu[:, n:])
        dg, du, _ = G.gated_act_mxfp8_grad(dh, c, s)
        return h, dg, du, G.ragged_dot_k(xc, dg, gs, lhs_scale=xs), G.mxfp8_dequantize(xc, xs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (4, 5, 6):
        x.copy_(rows(seed, m, k, BF)), gu.copy_(rows(seed + 10, m, 2 * n, BF)), dh.copy_(rows(seed + 20, m, n, BF))
        gs.copy_(torch.tensor([seed, 96 - seed], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_past_32_bits():
    """More than 2^32 codes: the last rows of a long checkpoint."""
    say("long")
    m, k = (1 << 32) // 4096 + 5, 4096
    tail = rows(8, 6, k, BF)
    x = torch.zeros(m, k, dtype=BF, device=DEV)
    x[-6:] = tail
    codes, scale = G.mxfp8_quantize(x)
    want_c, want_s = oracle.mxfp8_quantize(val(tail))
    assert np.array_equal(u8(codes[-6:]), want_c) and np.array_equal(u8(scale[-6:]), want_s)
    assert int(codes[:-6].view(torch.uint8).max()) == 0
    del x
    out = G.mxfp8_dequantize(codes, scale)
    assert np.array_equal(val(out[-6:]), oracle.mxfp8_values(want_c, want_s))
    n = k // 2
    h = torch.empty(m, n, dtype=BF, device=DEV)
    dg, du, h = G.gated_act_mxfp8_grad(out[:, :n].contiguous(), codes, scale, out=(None, None, h))
    v = oracle.mxfp8_values(want_c, want_s)
    check_h(h[-6:], v[:, :n], v[:, n:], "silu")
    h2, c2, s2 = G.gated_act_mxfp8(out[:, :n], out[:, n:], out=(h, None, None))
    # (not the same codes again: a largest value of 1.76 becomes 1.75, which the next smaller scale holds)
    want_c, want_s = oracle.mxfp8_quantize(v)
    assert np.array_equal(u8(c2[-6:]), want_c) and np.array_equal(u8(s2[-6:]), want_s)
    check_h(h2[-6:], v[:, :n], v[:, n:], "silu")
