"""GPU parity of the MXFP4 calls against the fp64 oracle.

Quantisation and its inverse are exact to the definition: codes, scale bytes and values are compared bit
for bit.  The product's bound: with exact 4-bit products, an fp32 accumulation of k terms is off by at most
one rounding (or truncation, 2^-23) per addition the hardware and the split make, fewer than k / 8 + 32,
each relative to the sum of magnitudes; a bf16 result adds half a step, 2^-8 of the value.
Outputs start out as NaN (or 0xAB bytes) and lie between guard rows that must not change.
"""
import numpy as np
import pytest
import torch

import oracle
from group_gemm_amd import _binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
GUARD = 64


def say(*a):
    print("[case]", *a, flush=True)


def guarded(shape, dtype, lead=GUARD):
    """A tensor of `shape` inside a larger buffer of marks; check(t) asserts that the marks stand."""
    n = int(np.prod(shape))
    fill = 0xAB if dtype == torch.uint8 else float("nan")
    buf = torch.full((n + 2 * lead,), fill, dtype=dtype, device=DEV)
    t = buf[lead:lead + n].view(shape)

    def check():
        ends = torch.cat([buf[:lead], buf[lead + n:]])
        assert (ends == 0xAB).all() if dtype == torch.uint8 else torch.isnan(ends.float()).all(), "wrote outside its output"
    return t, check


def host(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype in (B.FP4, torch.uint8) else t.double().cpu().numpy()


def same(got, want):
    return np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def rows_like(r, rows, k, dtype):
    """Values over many powers of two, with zero blocks, ties and values that saturate."""
    x = r.standard_normal((rows, k)) * 2.0 ** r.integers(-12, 12, (rows, k // 32)).repeat(32, axis=1)
    x[r.random((rows, k)) < 0.1] = 0.0
    x.reshape(rows, k // 32, 32)[r.random((rows, k // 32)) < 0.1] = 0.0
    ties = r.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.75, 6.0, -5.0, -0.25], (rows, k // 32, 32))
    ties[..., 0] = 7.0
    x = np.where((r.random((rows, k // 32)) < 0.3)[..., None], ties, x.reshape(rows, k // 32, 32)).reshape(rows, k)
    return torch.from_numpy(x).to(dtype).to(DEV)


def check_quantized(x, codes, scale):
    """bit-exact against the oracle of x's own values"""
    want_c, want_s = oracle.mxfp4_quantize(x.double().cpu().numpy())
    got_s, ok = host(scale), want_s != 255
    assert np.array_equal(got_s, oracle.mxfp4_panels(want_s)), "scale bytes"
    c = host(codes)
    keep = np.repeat(ok, 16, axis=-1)
    assert np.array_equal(c[keep], want_c[keep]), "codes"
    return want_s


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 4096), (3, 256), (33, 288), (24, 2880), (130, 992), (7, 7168)])
def test_quantize(rows, k, dtype):
    say("quantize", rows, k, dtype)
    x = rows_like(np.random.default_rng(rows + k), rows, k, dtype)
    c, cc = guarded((rows, k // 2), torch.uint8)
    s, sc = guarded((-(-k // 256), rows, 8), torch.uint8)
    B.mxfp4_quantize(x, out=(c, s))
    check_quantized(x, c, s)
    cc(), sc()
    c2, s2 = B.mxfp4_quantize(x)
    assert c2.dtype == B.FP4 and np.array_equal(host(c2), host(c)) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_strided_and_unaligned_rows(dtype):
    say("strided", dtype)
    big = rows_like(np.random.default_rng(1), 37, 640, dtype)
    for x in (big[:, 32:352], big[:, 3:323], big[5:6, 1:97], big[::2, 8:584]):
        check_quantized(x, *B.mxfp4_quantize(x))
    flat = torch.empty(33 * 96 + 1, dtype=dtype, device=DEV)[1:].view(33, 96)   # not 16-byte aligned
    flat.copy_(big[:33, :96])
    check_quantized(flat, *B.mxfp4_quantize(flat))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_extremes(dtype):
    say("extremes", dtype)
    t = torch.finfo(dtype)
    x = torch.zeros(12, 64, dtype=dtype, device=DEV)
    x[0, 3], x[1, 40], x[2, 0] = float("inf"), float("-inf"), float("nan")
    x[3, :] = t.max
    x[4, :] = t.min
    x[5, 5], x[5, 40] = t.tiny, t.smallest_normal * 4
    x[6, 9] = t.tiny / 8            # a subnormal
    x[7, :] = -0.0
    x[8, ::2] = 2.0 ** -126
    x[9, 33], x[9, 34] = t.max, 1.0
    x[10, :] = torch.linspace(-1, 1, 64)
    x[11, 3], x[11, 4] = float("nan"), float("inf")
    c, s = B.mxfp4_quantize(x)
    bytes_ = check_quantized(x, c, s)
    assert (bytes_[[0, 1, 2, 11]] == 255).sum() == 4
    for out_dtype in (BF, F32):
        v = B.mxfp4_dequantize(c, s, out_dtype=out_dtype)
        assert same(host(v), oracle.mxfp4_values(host(c), host(s)))
        assert torch.isnan(v[0, :32]).all() and not torch.isnan(v[0, 32:]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("g,k,n", [(1, 32, 1), (3, 288, 257), (2, 256, 256), (5, 64, 40), (2, 544, 1000), (1, 1024, 129), (4, 96, 7)])
def test_quantize_weights(g, k, n, dtype):
    say("weights", g, k, n, dtype)
    wt = rows_like(np.random.default_rng(k + n), g * n, k, dtype).view(g, n, k)
    w = wt.transpose(1, 2).contiguous()
    c, cc = guarded((g, n, k // 2), torch.uint8)
    s, sc = guarded((g, -(-k // 256), n, 8), torch.uint8)
    B.mxfp4_quantize_weights(w, out=(c, s))
    check_quantized(wt, c, s)
    cc(), sc()
    off = torch.empty(w.numel() + 1, dtype=dtype, device=DEV)[1:].view(g, k, n)   # not 16-byte aligned
    off.copy_(w)
    c2, s2 = B.mxfp4_quantize_weights(off)
    assert np.array_equal(host(c2), host(c)) and torch.equal(s2, s)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("g,n,k", [(0, 1, 32), (0, 65, 288), (0, 4, 7168), (3, 33, 544), (2, 256, 256), (1, 1, 96)])
def test_dequantize(g, n, k, out_dtype):
    """Every code under scale bytes from the whole range, NaN among them (g = 0: rows)."""
    say("dequantize", g, n, k, out_dtype)
    r = np.random.default_rng(g + n + k)
    lead = (g,) if g else ()
    codes = r.integers(0, 256, lead + (n, k // 2)).astype(np.uint8)
    scale = r.integers(0, 256, lead + (-(-k // 256), n, 8)).astype(np.uint8)
    out, check = guarded(lead + (n, k), out_dtype)
    B.mxfp4_dequantize(torch.from_numpy(codes).to(DEV), torch.from_numpy(scale).to(DEV), out=out)
    want = oracle.mxfp4_values(codes, scale)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)   # 3 and 6 times 2^127 and 2^128: infinite in both types
    assert same(host(out), want)
    check()
    off = torch.full((out.numel() + 1,), float("nan"), dtype=out_dtype, device=DEV)[1:].view(out.shape)
    B.mxfp4_dequantize(torch.from_numpy(codes).to(DEV), torch.from_numpy(scale).to(DEV), out=off)
    assert same(host(off), want)


def operands(r, m, k, n, g, pad=0):
    """Quantised normal rows and weights; the scale bytes past k are `pad`."""
    lc, ls = oracle.mxfp4_quantize(r.standard_normal((m, k)) * np.exp(r.standard_normal(k)))
    rc, rs = oracle.mxfp4_quantize(r.standard_normal((g, n, k)) / np.sqrt(max(k, 1)))
    lp, rp = oracle.mxfp4_panels(ls), oracle.mxfp4_panels(rs)
    if pad and k % 256:
        lp[-1, :, (k // 32) % 8:] = pad
        rp[:, -1, :, (k // 32) % 8:] = pad
    return lc, lp, rc, rp


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check_product(lc, lp, rc, rp, gs, out_dtype=BF, lead=GUARD, ws=None):
    m, n, k = lc.shape[0], rc.shape[1], 2 * lc.shape[1]
    out, guard = guarded((m, n), out_dtype, lead)
    B.ragged_dot_m_mxfp4(dev(lc), dev(rc), dev(np.asarray(gs, np.int32)), dev(lp), dev(rp), out=out, workspace=ws)
    want, mag = oracle.ragged_dot_m_mxfp4(lc, lp, rc, rp, gs)
    bound = (k / 8 + 32) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(want) if out_dtype == BF else 0)
    got = host(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) - bound)
    covered = min(m, sum(max(int(s), 0) for s in gs))
    assert not got[covered:].any(), "rows past the groups are 0"
    guard()
    return out


CASES = [
    # m, k, n, sizes
    (1, 32, 1, [1]),
    (1, 4096, 64, [0, 0, 1, 0]),
    (2, 4096, 200, [1, 0, 0, 0, 0, 1, 0, 0]),
    (5, 288, 33, [2, 0, 3]),
    (17, 2880, 100, [4, 13]),
    (64, 544, 256, [1, 0, 30, 16, 17]),
    (70, 256, 257, [33, 0, 31]),
    (100, 1024, 48, [100]),
    (130, 96, 20, [127, 0, 0]),
    (300, 512, 264, [0, 257, 0, 43]),
    (513, 1056, 520, [513]),
    (600, 768, 300, [255, 1, 256, 20, 60]),
    (21, 7168, 70, [9, 0, 11]),
    (8, 7168, 530, [1, 5, 2]),
    (40, 4128, 1100, [16, 0, 23, 1]),
    (3, 16384, 40, [1, 2]),
    (2, 64, 4000, [0, 1, 0, 0, 1]),
]


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_product(case, out_dtype):
    m, k, n, gs = CASES[case]
    say("product", m, k, n, gs, out_dtype)
    lc, lp, rc, rp = operands(np.random.default_rng(case), m, k, n, len(gs))
    check_product(lc, lp, rc, rp, gs, out_dtype)


TILES = [
    # long groups: whole tiles, partly filled ones, k of three panels and more, with and without a part panel
    (1000, 768, 512, [1000], BF),
    (1000, 1056, 511, [256, 500, 0, 31, 213], BF),
    (700, 2880, 96, [130, 470, 90], BF),
    (700, 544, 260, [700], F32),
    (2700, 1024, 6000, [2560, 0, 140], BF),          # more tiles than compute units: several a workgroup
    (5000, 800, 2100, [1, 1024, 77, 1500, 0, 33, 300, 2000], F32),
    (300, 7168, 300, [290], BF),
]


@pytest.mark.parametrize("case", range(len(TILES)))
def test_product_tiles(case):
    m, k, n, gs, out_dtype = TILES[case]
    say("tiles", TILES[case])
    check_product(*operands(np.random.default_rng(70 + case), m, k, n, len(gs)), gs, out_dtype)


def test_product_tiles_of_many_groups():
    say("tiles of many groups")
    r = np.random.default_rng(80)
    gs = r.integers(0, 110, 300)
    gs[r.random(300) < 0.1] = 0
    lc, lp, rc, rp = operands(r, int(gs.sum()) + 40, 800, 24, 300)
    check_product(lc, lp, rc, rp, gs)


@pytest.mark.parametrize("tokens", [3, 40, 700])
@pytest.mark.parametrize("g", [65, 300, 1024])
def test_product_many_groups(g, tokens):
    say("many groups", g, tokens)
    r = np.random.default_rng(g + tokens)
    gs = np.bincount(r.integers(0, g, tokens), minlength=g)
    lc, lp, rc, rp = operands(r, tokens + 3, 160, 24, g)
    check_product(lc, lp, rc, rp, gs)


def test_product_scale_bytes_past_k_are_ignored():
    say("padding bytes")
    for m, k, n, gs in ((9, 96, 40, [4, 5]), (600, 288, 272, [300, 300])):
        a = check_product(*operands(np.random.default_rng(3), m, k, n, len(gs)), gs)
        b = check_product(*operands(np.random.default_rng(3), m, k, n, len(gs), pad=255), gs)
        assert torch.equal(a, b)


@pytest.mark.parametrize("m", [10, 400])
def test_product_nan_scale_stays_in_its_row_and_column(m):
    say("nan scale", m)
    k, n, gs = 512, 72, [m // 2, m - m // 2]
    lc, lp, rc, rp = operands(np.random.default_rng(4), m, k, n, 2)
    want, _ = oracle.ragged_dot_m_mxfp4(lc, lp, rc, rp, gs)
    lp[1, 3, 5] = 255        # row 3 (group 0)
    rp[1, 0, 17, 2] = 255    # column 17 of group 1
    out = host(B.ragged_dot_m_mxfp4(dev(lc), dev(rc), dev(np.asarray(gs, np.int32)), dev(lp), dev(rp)))
    nan = np.zeros((m, n), bool)
    nan[3] = True
    nan[gs[0]:, 17] = True
    assert np.array_equal(np.isnan(out), nan)
    assert np.allclose(out[~nan], want[~nan], rtol=2.0 ** -7, atol=1e-2)


@pytest.mark.parametrize("m", [9, 300])
def test_product_bad_sizes(m):
    say("bad sizes", m)
    lc, lp, rc, rp = operands(np.random.default_rng(5), m, 256, 40, 4)
    for gs, flags in (([3, -2, 4, 1], B.DEV_NEGATIVE_SIZE), ([m, 7, 0, m], B.DEV_SUM_EXCEEDS_M), ([0, 0, 0, 0], 0),
                      ([-5, 2 ** 31 - 1, 2 ** 31 - 1, 3], B.DEV_NEGATIVE_SIZE | B.DEV_SUM_EXCEEDS_M)):
        ws = torch.full((B.workspace_bytes("ragged_m", m, 256, 40, 4, 0, B.FP4),), 0xAB, dtype=torch.uint8, device=DEV)
        check_product(lc, lp, rc, rp, gs, ws=ws)
        assert B.read_device_status(ws) == flags


def test_product_unaligned_output_and_empty_shapes():
    say("unaligned output, empty shapes")
    for m, n in ((20, 64), (300, 264)):
        for dt in (BF, F32):
            check_product(*operands(np.random.default_rng(6), m, 256, n, 2), [m // 2, 3], dt, lead=65)
    for m, k, n in ((0, 64, 8), (4, 64, 0), (4, 0, 8)):
        lc, lp, rc, rp = np.zeros((m, k // 2), np.uint8), np.zeros((-(-k // 256), m, 8), np.uint8), np.zeros((2, n, k // 2), np.uint8), np.zeros((2, -(-k // 256), n, 8), np.uint8)
        out = B.ragged_dot_m_mxfp4(dev(lc), dev(rc), dev(np.array([2, 2], np.int32)), dev(lp), dev(rp))
        assert out.shape == (m, n) and not out.any()


def test_product_does_not_depend_on_the_other_rows():
    """A row's result is the same bits alone and in a batch handled by the same kernel."""
    say("row alone")
    lc, lp, rc, rp = operands(np.random.default_rng(8), 12, 1312, 48, 4)
    full = B.ragged_dot_m_mxfp4(dev(lc), dev(rc), dev(np.array([3, 3, 3, 3], np.int32)), dev(lp), dev(rp), out_dtype=F32)
    one = B.ragged_dot_m_mxfp4(dev(lc[7:8]), dev(rc), dev(np.array([0, 0, 1, 0], np.int32)), dev(lp[:, 7:8]), dev(rp), out_dtype=F32)
    assert torch.equal(full[7:8], one)


def test_permute_of_mxfp4_rows():
    say("permute")
    r = np.random.default_rng(9)
    for tokens, top_k, k, g in ((1, 2, 32, 8), (37, 3, 288, 5), (300, 8, 2880, 64), (513, 1, 4096, 7)):
        codes, scale = oracle.mxfp4_quantize(r.standard_normal((tokens, k)))
        experts = r.integers(-1, g + 1, (tokens, top_k)).astype(np.int32)   # some ids are not routed
        sx, ss, gs, s2c, c2s = B.moe_permute(dev(codes).view(B.FP4), dev(experts), g, x_scale=dev(oracle.mxfp4_panels(scale)))
        ox, os_, ogs, os2c, oc2s = oracle.moe_permute(codes, experts, g, scale)
        assert np.array_equal(host(sx), ox) and np.array_equal(host(ss), oracle.mxfp4_panels(os_))
        assert np.array_equal(gs.cpu().numpy(), ogs) and np.array_equal(s2c.cpu().numpy(), os2c) and np.array_equal(c2s.cpu().numpy(), oc2s)


def test_binding_refusals():
    say("refusals")
    x = torch.zeros(8, 64, dtype=BF, device=DEV)
    c, s = B.mxfp4_quantize(x)
    w = torch.zeros(2, 16, 32, dtype=torch.uint8, device=DEV).view(B.FP4)
    wsc = torch.zeros(2, 1, 16, 8, dtype=torch.uint8, device=DEV)
    gs = torch.tensor([4, 4], dtype=torch.int32, device=DEV)
    assert B.ragged_dot_m_mxfp4(c, w, gs, s, wsc).shape == (8, 16)
    for bad in (lambda: B.mxfp4_quantize(x[:, :48]), lambda: B.mxfp4_quantize(x.half()), lambda: B.mxfp4_quantize(x.t()),
                lambda: B.mxfp4_quantize(x[:1].expand(4, 64)), lambda: B.mxfp4_quantize(x[0]),
                lambda: B.mxfp4_quantize(x, out=(c[:4], None)), lambda: B.mxfp4_quantize(x, out=(None, s[:, :4])),
                lambda: B.mxfp4_quantize_weights(x), lambda: B.mxfp4_quantize_weights(torch.zeros(2, 40, 8, device=DEV)),
                lambda: B.mxfp4_quantize_weights(torch.zeros(2, 8, 64, device=DEV).transpose(1, 2)),
                lambda: B.mxfp4_dequantize(c, s[:, :4]), lambda: B.mxfp4_dequantize(x, s), lambda: B.mxfp4_dequantize(c, s, out_dtype=torch.float16, out=x),
                lambda: B.ragged_dot_m_mxfp4(c, w, gs, wsc, s), lambda: B.ragged_dot_m_mxfp4(c, w, gs.long(), s, wsc),
                lambda: B.ragged_dot_m_mxfp4(c, w[..., :16], gs, s, wsc), lambda: B.ragged_dot_m_mxfp4(c, w, gs[:1], s, wsc),
                lambda: B.ragged_dot_m_mxfp4(c, w, gs, s, wsc, out=torch.zeros(8, 17, dtype=BF, device=DEV)),
                lambda: B.ragged_dot_m_mxfp4(c, w, gs, s, wsc, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)),
                lambda: B.moe_permute(c, torch.zeros(8, 2, dtype=torch.int32, device=DEV), 4),
                lambda: B.moe_permute(c, torch.zeros(8, 2, dtype=torch.int32, device=DEV), 4, x_scale=s[:, :4])):
        with pytest.raises(ValueError):
            bad()


def test_layer_on_another_stream_and_in_a_graph():
    """quantise -> permute -> product -> un-permute as one serving step: on a side stream, then captured and
    replayed over new tokens and routing, each replay equal to the eager step, eager work in between."""
    say("layer: side stream and graph")
    tokens, top_k, g, k, n = 50, 2, 8, 288, 264
    r = np.random.default_rng(10)
    w, ws = B.mxfp4_quantize_weights(dev(r.standard_normal((g, k, n)) / np.sqrt(k)).to(BF))
    x = torch.zeros(tokens, k, dtype=BF, device=DEV)
    experts = torch.zeros(tokens, top_k, dtype=torch.int32, device=DEV)
    rw = torch.zeros(tokens, top_k, device=DEV)

    def fill(seed):
        q = np.random.default_rng(seed)
        x.copy_(dev(q.standard_normal((tokens, k))).to(BF))
        experts.copy_(dev(q.integers(0, g, (tokens, top_k)).astype(np.int32)))
        rw.copy_(dev(q.random((tokens, top_k)).astype(np.float32)))

    def step():
        c, s = B.mxfp4_quantize(x)
        sc, ss, gs, _, c2s = B.moe_permute(c, experts, g, x_scale=s)
        return B.moe_unpermute(B.ragged_dot_m_mxfp4(sc, w, gs, ss, ws), c2s, rw)

    fill(0)
    eager = step()
    # the step against the oracle, from the library's own codes
    c, s = B.mxfp4_quantize(x)
    oc, os_ = oracle.mxfp4_quantize(x.double().cpu().numpy())
    ox, osc, ogs, _, oc2s = oracle.moe_permute(oc, experts.cpu().numpy(), g, os_)
    y, mag = oracle.ragged_dot_m_mxfp4(ox, oracle.mxfp4_panels(osc), host(w), host(ws), ogs)
    # each row of y is off by its own bound (above); un-permute adds at most top_k terms and rounds once more
    yb = (k / 8 + 32) * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(y)
    wn = rw.double().cpu().numpy()
    want = oracle.moe_unpermute(y.astype(np.float64), oc2s, wn)
    bound = oracle.moe_unpermute(yb, oc2s, wn) * 1.01 + 2.0 ** -7.9 * np.abs(want)
    assert (np.abs(host(eager) - want) <= bound).all()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, eager)

    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            captured = step()
    for seed in range(1, 5):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, step()), seed


LONG = [
    # some thousands of rows in long groups and wide enough for the 256 x 256 tiles: widths that whole stores divide and
    # widths that they do not (a last piece of one to seven elements), k with and without a part panel, odd row counts
    (1701, 544, 4997, [1000, 0, 640, 20], BF),
    (1701, 544, 4997, [1000, 0, 640, 20], F32),
    (1700, 800, 5000, [801, 799, 100], BF),
    (1703, 608, 5004, [1, 1702], F32),
    (1703, 1056, 5003, [1100, 602], F32),
    (5000, 800, 4103, [1, 1024, 77, 1500, 0, 33, 300, 2000], BF),
    (2304, 1312, 4098, [256, 512, 768, 700], BF),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_product_long_groups(case):
    m, k, n, gs, out_dtype = LONG[case]
    say("long groups", LONG[case])
    check_product(*operands(np.random.default_rng(90 + case), m, k, n, len(gs)), gs, out_dtype)


def test_product_long_groups_bad_sizes_and_nan_scales():
    say("long groups: bad sizes, nan scales")
    m, k, n = 1700, 800, 5000
    lc, lp, rc, rp = operands(np.random.default_rng(100), m, k, n, 3, pad=255)
    for gs, flags in (([900, -2, 700], B.DEV_NEGATIVE_SIZE), ([m, 7, m], B.DEV_SUM_EXCEEDS_M), ([0, 0, 0], 0)):
        ws = torch.full((B.workspace_bytes("ragged_m", m, k, n, 3, 0, B.FP4),), 0xAB, dtype=torch.uint8, device=DEV)
        check_product(lc, lp, rc, rp, gs, ws=ws)
        assert B.read_device_status(ws) == flags
    gs = [900, 0, 790]
    lp[1, 3, 5] = 255        # row 3 (group 0)
    rp[2, 3, 17, 0] = 255    # column 17 of group 2, in the part panel
    out = host(B.ragged_dot_m_mxfp4(dev(lc), dev(rc), dev(np.asarray(gs, np.int32)), dev(lp), dev(rp)))
    nan = np.zeros((m, n), bool)
    nan[3] = True
    nan[900:1690, 17] = True
    assert np.array_equal(np.isnan(out), nan)


@pytest.mark.parametrize("n", [1, 5, 115, 129, 1025])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_product_narrow_and_ragged_widths(n, out_dtype):
    """One column tile or a few, many row tiles of many groups; some tens of rows and several row tiles a group."""
    say("narrow", n, out_dtype)
    r = np.random.default_rng(n)
    for g, most in ((40, 60), (5, 300), (3, 5)):
        gs = r.integers(0, most, g)
        m = int(gs.sum()) + 9
        check_product(*operands(r, m, 352, n, g), gs, out_dtype)


def test_empty_quantisation():
    say("empty")
    for rows, k in ((0, 64), (3, 0)):
        c, s = B.mxfp4_quantize(torch.zeros(rows, k, device=DEV))
        assert c.shape == (rows, k // 2) and s.shape == (-(-k // 256), rows, 8)
        assert B.mxfp4_dequantize(c, s).shape == (rows, k)
    for g, k, n in ((2, 0, 5), (2, 64, 0)):
        c, s = B.mxfp4_quantize_weights(torch.zeros(g, k, n, device=DEV))
        assert c.shape == (g, n, k // 2) and s.shape == (g, -(-k // 256), n, 8)
        assert B.mxfp4_dequantize(c, s).shape == (g, n, k)


@pytest.mark.parametrize("m,k,n,g", [(3, 2880, 1000001, 4), (3, 65536, 50000, 4), (40, 65536, 50000, 4), (1700, 65536, 50000, 4)])
def test_product_of_weights_past_32_bits(m, k, n, g):
    """The last group's codes begin past 4 GiB; eight rows and some columns against 64 bits."""
    say("large weights", m, k, n, g)
    gen = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randint(0, 256, (g, n, k // 2), dtype=torch.uint8, device=DEV, generator=gen)
    ws = torch.randint(116, 124, (g, -(-k // 256), n, 8), dtype=torch.uint8, device=DEV, generator=gen)
    assert (g - 1) * n * (k // 2) > 2 ** 32
    x = torch.randint(0, 256, (m, k // 2), dtype=torch.uint8, device=DEV, generator=gen)
    xs = torch.randint(116, 124, (-(-k // 256), m, 8), dtype=torch.uint8, device=DEV, generator=gen)
    if k % 256:
        ws[:, -1, :, k % 256 // 32:] = 0
        xs[-1, :, k % 256 // 32:] = 0
    gs = torch.tensor([0] * (g - 1) + [m], dtype=torch.int32, device=DEV)
    out = B.ragged_dot_m_mxfp4(x, w, gs, xs, ws, out_dtype=F32)
    rows = torch.tensor(sorted({0, 1, 2, m // 2, m - 3, m - 2, m - 1}), device=DEV)
    cols = torch.tensor([0, 1, 17, n // 2, n - 300, n - 2, n - 1], device=DEV)
    a = oracle.mxfp4_values(host(x[rows]), host(xs[:, rows]))
    b = oracle.mxfp4_values(host(w[-1, cols]), host(ws[-1][:, cols]))
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    assert (np.abs(host(out[rows][:, cols]) - want) <= (k / 8 + 32) * 2.0 ** -23 * mag).all()


def test_quantisation_past_32_bits():
    """More than 2^32 elements: the last rows are quantised and put back as they are alone."""
    say("large rows")
    rows, k = 70001, 65536
    x = torch.empty(rows, k, dtype=BF, device=DEV)
    x[:-3] = 0
    tail = torch.randn(3, k, device=DEV).to(BF)
    x[-3:] = tail
    c, s = B.mxfp4_quantize(x)
    c3, s3 = B.mxfp4_quantize(tail)
    assert torch.equal(c[-3:].view(torch.uint8), c3.view(torch.uint8)) and torch.equal(s[:, -3:], s3)
    assert not c[:-3].view(torch.uint8).any()
    del x
    assert torch.equal(B.mxfp4_dequantize(c, s)[-3:], B.mxfp4_dequantize(c3, s3))


def test_two_streams_and_one_workspace():
    """The workspace holds a status word only: calls on two streams may share it, and so may captured graphs."""
    say("two streams, one workspace")
    r = np.random.default_rng(20)
    ws = torch.zeros(B.workspace_bytes("ragged_m", 600, 544, 700, 3, 0, B.FP4), dtype=torch.uint8, device=DEV)
    calls, wants = [], []
    for m, gs in ((600, [300, 0, 290]), (9, [3, 3, 3])):
        lc, lp, rc, rp = (dev(a) for a in operands(r, m, 544, 700, 3))
        sizes = dev(np.asarray(gs, np.int32))
        calls.append(lambda lc=lc, lp=lp, rc=rc, rp=rp, sizes=sizes: B.ragged_dot_m_mxfp4(lc, rc, sizes, lp, rp, workspace=ws))
        wants.append(calls[-1]())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(calls[i]())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, wants[i]) for o in outs[i])
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            o = calls[i]()
        graphs.append((g, o))
    for _ in range(3):
        for (g, o), want in zip(graphs, wants):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(calls[0](), wants[0])
