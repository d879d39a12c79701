"""GPU tests of the low-rank adapters and their gradients against the fp64 oracle.

Bounds.  A sum of N products is off by (N + 40) 2^-24 of the sum of their magnitudes, in whatever order.  bf16 operands
meet the fp32 v (or u) as two bf16 values: half a step of the second is 2^-8 of what the first, 2^-8 off, left, 2^-16 in all;
as three, in row sums that leave in fp32, 2^-24.  A result adds half a step of its type: 2^-8 (bf16) or 2^-24 of its value.
"""
import numpy as np
import pytest
import torch

import group_gemm_amd as G
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24


def say(*a):
    print("[case]", *a, flush=True)


def val(t):
    return t.double().cpu().numpy()


def half(t):
    return {BF: 2.0 ** -8, F32: E}[t]


def rand(r, shape, dtype, scale=1.0):
    return torch.from_numpy((scale * r.standard_normal(shape)).astype(np.float32)).to(dtype).to(DEV)


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def framed(shape, dtype, pitch=None):
    """A tensor (rows `pitch` apart) in a buffer of a known pattern, and a check that the rest kept it."""
    shape = tuple(shape)
    size = torch.empty((), dtype=dtype).element_size()
    if pitch is None or len(shape) != 2:
        n = int(np.prod(shape))
        buf = torch.full(((n + 128) * size,), 0xA5, dtype=torch.uint8, device=DEV)
        t = buf[64 * size:(64 + n) * size].view(dtype).view(shape)
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[64 * size:(64 + n) * size] = False
    else:
        buf = torch.full((shape[0] + 2, pitch * size), 0xA5, dtype=torch.uint8, device=DEV)
        t = buf.view(dtype)[1:-1, 1:1 + shape[1]]
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[1:-1, size:(1 + shape[1]) * size] = False

    def check():
        assert bool((buf[mask] == 0xA5).all()), "wrote outside its output"
    return t, check


def within(got, want, bound, what=""):
    off = ~(np.abs(got - want) <= bound)
    i = tuple(np.argwhere(off)[0]) if off.any() else None
    assert i is None, f"{what}: {int(off.sum())} of {off.size} off, first {i}: {got[i]!r}, not {want[i]!r}, bound {bound[i]!r}"


def bounds(x, a, b, rows, scaling, out_dtype, bf16, want, base=None):
    """Bounds on v and out."""
    (m, k), (g, n, r) = x.shape, b.shape
    ev, eo = np.zeros((m, r)), np.zeros((m, n))
    for i, h in enumerate(rows):
        if 0 <= h < g:
            s = 1.0 if scaling is None else abs(float(scaling[h]))
            v, mag = np.abs(a[h] @ x[i]), np.abs(a[h]) @ np.abs(x[i])
            ev[i] = (k + 40) * E * mag
            ab = np.abs(b[h])
            eo[i] = s * (ab @ ev[i]) + ((2.0 ** -16 if bf16 else 0) + (2 * r + 40) * E) * s * (ab @ (v + ev[i]))
    if base is not None:
        eo += E * np.abs(base)
    return ev, eo + half(out_dtype) * 1.01 * (np.abs(want) + eo)


# m, k, n, r, sizes: one row; ranks of every width, odd ones; a border of every tile; groups without rows; rows past the last one;
# widths without any alignment; widths below a piece
SORTED = [(1, 32, 16, 1, [1]), (1, 4096, 520, 16, [0, 1]), (5, 64, 8, 4, [0, 5, 0]), (77, 129, 130, 11, [30, 1, 40]), (130, 256, 264, 16, [64, 65, 1]),
          (200, 515, 77, 32, [30, 0, 100, 33]), (300, 192, 1447, 64, [300]), (65, 1030, 515, 100, [33, 32]), (150, 320, 264, 128, [150]),
          (40, 640, 129, 200, [7, 33]), (100, 7, 3, 5, [50, 50]), (90, 2880, 96, 24, [40, 9]), (33, 64, 64, 16, [-4, 40]), (600, 256, 256, 8, [2] * 300),
          (20, 0, 24, 8, [20]), (20, 64, 0, 8, [20]), (257, 200, 300, 256, [250, 7]), (190, 128, 640, 40, [180, 10])]


def make(seed, m, k, n, r, g, dtype):
    rng = np.random.default_rng(seed)
    x = rand(rng, (m, k), dtype)
    a, b = rand(rng, (g, r, k), dtype, max(k, 1) ** -0.5), rand(rng, (g, n, r), dtype, r ** -0.5)
    return rng, x, a, b, torch.from_numpy(rng.uniform(0.25, 2, g).astype(np.float32)).to(DEV)


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("case", range(len(SORTED)))
def test_sorted_rows(case, types):
    m, k, n, r, sizes = SORTED[case]
    say("sorted", SORTED[case][:4], types)
    g = len(sizes)
    rng, x, a, b, s = make(case, m, k, n, r, g, types[0])
    base = rand(rng, (m, n), types[1])
    out, c1 = framed((m, n), types[1])
    v, c2 = framed((m, r), F32)
    ws = torch.empty(G.workspace_bytes("lora", m, k, n, g, r, types[0]), dtype=torch.uint8, device=DEV)
    G.ragged_lora(x, a, b, ints(sizes), base=base, scaling=s, v=v, out=out, workspace=ws)
    c1(), c2()
    rows = oracle.row_groups(sizes, m)
    want, wv = oracle.ragged_lora(val(x), val(a), val(b), rows, val(s), val(base))
    ev, eo = bounds(val(x), val(a), val(b), rows, val(s), types[1], types[0] == BF, want, val(base))
    within(val(v), wv, ev, "v")
    within(val(out), want, eo, "out")
    none = torch.from_numpy(rows < 0).to(DEV)
    assert torch.equal(out[none], base[none]) and not bool(v[none].any())
    assert G.read_device_status(ws) == (1 if min(sizes) < 0 else 0) | (2 if sum(max(z, 0) for z in sizes) > m else 0)


# m, k, n, r, g, chance of none: fewer rows than adapters and more, one adapter, several chunks of rows
ANY = [(1, 64, 40, 16, 1, 0.0), (1, 1024, 520, 16, 8, 0.0), (3, 65, 33, 5, 1024, 0.3), (96, 512, 264, 32, 64, 0.1), (300, 192, 130, 8, 3, 0.5), (700, 128, 77, 16, 1, 0.2),
       (1300, 96, 40, 4, 5, 0.0), (2100, 64, 72, 64, 70, 0.1), (40, 256, 300, 120, 2, 1.0), (64, 320, 64, 256, 9, 0.1),
       (700, 128, 80, 16, 2, 0.3), (1500, 256, 264, 64, 3, 0.1), (1100, 131, 520, 32, 1, 0.5), (600, 75, 40, 128, 2, 0.0), (500, 64, 1032, 256, 1, 0.2)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(ANY)))
def test_rows_in_any_order(case, dtype):
    m, k, n, r, g, none = ANY[case]
    say("any order", ANY[case], dtype)
    rng, x, a, b, s = make(100 + case, m, k, n, r, g, dtype)
    rows = rng.integers(0, g, m)
    rows[rng.random(m) < none] = -1
    if m > 4:
        rows[[1, 3]] = [g, -(1 << 31)]                     # none of the adapters
    base = rand(rng, (m, n), dtype)
    out, c1 = framed((m, n), dtype)
    v, c2 = framed((m, r), F32)
    G.ragged_lora(x, a, b, row_group=ints(rows), base=base, scaling=s, v=v, out=out)
    c1(), c2()
    want, wv = oracle.ragged_lora(val(x), val(a), val(b), rows, val(s), val(base))
    ev, eo = bounds(val(x), val(a), val(b), rows, val(s), dtype, dtype == BF, want, val(base))
    within(val(v), wv, ev, "v")
    within(val(out), want, eo, "out")
    left = torch.from_numpy((rows < 0) | (rows >= g)).to(DEV)
    assert torch.equal(out[left], base[left]) and not bool(v[left].any())


@pytest.mark.parametrize("any_order", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_in_place_no_base_no_scaling(dtype, any_order):
    say("strides", dtype, any_order)
    m, k, n, r, g = 70, 130, 201, 12, 4
    rng, x, a, b, s = make(7, m, k, n, r, g, dtype)
    rows = oracle.row_groups([20, 0, 30, 10], m)
    pick = dict(row_group=ints(rows)) if any_order else dict(group_sizes=ints([20, 0, 30, 10]))
    plain = G.ragged_lora(x, a, b, scaling=s, **pick)
    want, _ = oracle.ragged_lora(val(x), val(a), val(b), rows, val(s))
    _, eo = bounds(val(x), val(a), val(b), rows, val(s), dtype, dtype == BF, want)
    within(val(plain), want, eo)
    assert not bool(plain[60:].any())
    assert torch.equal(G.ragged_lora(x, a, b, scaling=torch.ones(g, device=DEV), **pick), G.ragged_lora(x, a, b, **pick))
    wide = torch.empty(m, k + 5, dtype=dtype, device=DEV)
    wide[:, 3:k + 3] = x
    base = rand(rng, (m, n), dtype)
    dense = G.ragged_lora(x, a, b, base=base, scaling=s, **pick)
    out, check = framed((m, n), dtype, pitch=n + 6)
    out.copy_(base)
    G.ragged_lora(wide[:, 3:k + 3], a, b, base=out, out=out, scaling=s, **pick)
    check()
    assert torch.equal(out, dense)
    both = torch.zeros(m, 2 * n, dtype=dtype, device=DEV)      # one matrix's halves: base and out interleave
    both[:, :n] = base
    G.ragged_lora(x, a, b, base=both[:, :n], out=both[:, n:], scaling=s, **pick)
    assert torch.equal(both, torch.cat([base, dense], 1))


@pytest.mark.parametrize("any_order", [False, True])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32)])
def test_whole_lines_in_place_strided_and_without_base(types, any_order):
    """Many rows an adapter and widths of whole 16 bytes, with rows without an adapter: as above."""
    say("lines", types, any_order)
    m, k, n, r, g = 400, 128, 264, 24, 3
    rng, x, a, b, s = make(17, m, k, n, r, g, types[0])
    rows = oracle.row_groups([200, 0, 120], m)
    pick = dict(row_group=ints(rows)) if any_order else dict(group_sizes=ints([200, 0, 120]))
    plain = G.ragged_lora(x, a, b, scaling=s, out_dtype=types[1], **pick)
    want, _ = oracle.ragged_lora(val(x), val(a), val(b), rows, val(s))
    _, eo = bounds(val(x), val(a), val(b), rows, val(s), types[1], True, want)
    within(val(plain), want, eo)
    assert not bool(plain[320:].any())
    base = rand(rng, (m, n), types[1])
    dense = G.ragged_lora(x, a, b, base=base, scaling=s, **pick)
    want, _ = oracle.ragged_lora(val(x), val(a), val(b), rows, val(s), val(base))
    _, eo = bounds(val(x), val(a), val(b), rows, val(s), types[1], True, want, val(base))
    within(val(dense), want, eo)
    wide = torch.full((m, 3 * n), float("nan"), dtype=types[1], device=DEV)
    out = wide[:, n:2 * n]
    out.copy_(base)
    G.ragged_lora(x, a, b, base=out, out=out, scaling=s, **pick)
    assert torch.equal(out, dense) and bool(wide[:, :n].isnan().all()) and bool(wide[:, 2 * n:].isnan().all())
    both = torch.zeros(m, 2 * n, dtype=types[1], device=DEV)
    both[:, :n] = base
    G.ragged_lora(x, a, b, base=both[:, :n], out=both[:, n:], scaling=s, **pick)
    assert torch.equal(both, torch.cat([base, dense], 1))


@pytest.mark.parametrize("any_order", [False, True])
@pytest.mark.parametrize("wide", [1, 8])
def test_values_of_other_rows_and_adapters(any_order, wide):
    """An adapter of NaN and infinities, rows of NaN and a base of NaN stay where they belong."""
    say("non-finite", any_order, wide)
    m, k, n, r, g = 90 * wide, 200, 136, 16, 5
    sizes = [20 * wide, 15 * wide, 20 * wide, 0, 20 * wide]
    rng, x, a, b, s = make(8, m, k, n, r, g, BF)
    rows = rng.permutation(oracle.row_groups(sizes, m)) if any_order else oracle.row_groups(sizes, m)
    pick = dict(row_group=ints(rows)) if any_order else dict(group_sizes=ints(sizes))
    base = rand(rng, (m, n), BF)
    good = G.ragged_lora(x, a, b, base=base, scaling=s, **pick)
    a[1], b[3], b[1, 0] = float("nan"), float("inf"), float("inf")
    a[3] = float("nan")
    at = int(np.argwhere(rows == 2)[3, 0])
    x[at] = float("nan")
    x[torch.from_numpy(rows < 0).to(DEV)] = float("nan")
    base[int(np.argwhere(rows == 0)[2, 0]), 5] = float("nan")
    got = G.ragged_lora(x, a, b, base=base, scaling=s, **pick)
    bad = np.zeros((m, n), bool)
    bad[rows == 1] = True
    bad[at] = True
    bad[int(np.argwhere(rows == 0)[2, 0]), 5] = True
    assert np.array_equal(np.isnan(val(got)), bad)
    assert torch.equal(got[torch.from_numpy(~bad).to(DEV)], good[torch.from_numpy(~bad).to(DEV)])


@pytest.mark.parametrize("any_order", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("wide", [1, 10])
@pytest.mark.parametrize("knr", [(131, 77, 11), (75, 264, 24), (128, 264, 40), (515, 131, 100), (192, 72, 3)])
def test_non_finite_neighbours_at_odd_sizes(knr, wide, dtype, any_order):
    """What lies behind a row's end, a rank's end and a column's weights is another row's, adapter's or column's."""
    say("non-finite odd", knr, wide, dtype, any_order)
    k, n, r = knr
    sizes, m = [13 * wide, 9 * wide, 11 * wide], 37 * wide
    rng, x, a, b, s = make(18, m, k, n, r, 3, dtype)
    rows = rng.permutation(oracle.row_groups(sizes, m)) if any_order else oracle.row_groups(sizes, m)
    pick = dict(row_group=ints(rows)) if any_order else dict(group_sizes=ints(sizes))
    base = rand(rng, (m, n), dtype)
    good = G.ragged_lora(x, a, b, base=base, scaling=s, **pick)
    bad = np.zeros((m, n), bool)
    a[1], b[1] = float("nan"), float("inf")                # the adapter behind the first and before the last
    bad[rows == 1] = True
    at = np.flatnonzero(rows != 1)[::3]                    # rows of infinities beside rows without
    x[torch.from_numpy(at).to(DEV)] = float("inf")
    bad[at] = True
    bad[rows < 0] = False
    for c in (0, n // 2, n - 1):                           # whole columns of infinities
        b[0, c], b[2, c] = float("inf"), float("nan")
        bad[(rows == 0) | (rows == 2), c] = True
    got = G.ragged_lora(x, a, b, base=base, scaling=s, **pick)
    ok = torch.from_numpy(~bad).to(DEV)
    assert bool(ok.any()) and torch.equal(got[ok], good[ok])
    assert not np.isfinite(val(got)[bad]).any()


def test_same_result_twice_and_sorted_as_in_any_order():
    say("twice")
    m, k, n, r, g = 500, 1024, 640, 16, 3
    rng, x, a, b, s = make(9, m, k, n, r, g, BF)
    base = rand(rng, (m, n), F32)
    first = G.ragged_lora(x, a, b, ints([200, 0, 290]), base=base, scaling=s)
    for _ in range(3):
        assert torch.equal(first, G.ragged_lora(x, a, b, ints([200, 0, 290]), base=base, scaling=s))
    other = G.ragged_lora(x, a, b, row_group=ints(oracle.row_groups([200, 0, 290], m)), base=base, scaling=s)
    assert float((first - other).abs().max()) <= 1e-5 * float(first.abs().max())


# ---------------------------------------------------------------------------------------------------------------
# gradients

# m, k, n, r, sizes: as above, and groups of several chunks
GRADS = [(1, 32, 16, 1, [1]), (5, 64, 8, 4, [0, 5, 0]), (77, 160, 130, 11, [30, 1, 40]), (130, 256, 264, 16, [64, 65, 1]), (200, 544, 77, 32, [30, 0, 100, 33]),
         (65, 1024, 515, 100, [33, 32]), (150, 320, 264, 128, [150]), (40, 640, 129, 200, [7, 33]), (100, 32, 3, 5, [50, 50]), (33, 64, 64, 16, [-4, 40]),
         (1500, 96, 136, 8, [700, 0, 600]), (600, 64, 72, 4, [2] * 300), (700, 288, 40, 64, [699, 1]), (20, 0, 24, 8, [20]), (20, 64, 0, 8, [20]), (0, 32, 40, 8, [0, 3]),
         (530, 160, 200, 256, [530])]


def check_grads(got, x, v, dout, a, b, rows, s, dbase, dtype, gdtype, need_dx=True):
    (m, k), (g, n, r) = x.shape, b.shape
    dx, da, db = oracle.ragged_lora_grad(x, v, dout, a, b, rows, s, dbase)
    two = 2.0 ** -16 if dtype == BF else 0
    row_split = two if gdtype == BF else (2 * E if dtype == BF else 0)
    eu, u = np.zeros((m, r)), np.zeros((m, r))
    edx = np.zeros((m, k))
    eda, edb = np.zeros(da.shape), np.zeros(db.shape)
    for i, h in enumerate(rows):
        if 0 <= h < g:
            w = abs(float(s[h]))
            u[i], eu[i] = w * np.abs(dout[i] @ b[h]), w * (n + 40) * E * (np.abs(dout[i]) @ np.abs(b[h]))
            edx[i] = eu[i] @ np.abs(a[h]) + (two + (2 * r + 40) * E) * ((u[i] + eu[i]) @ np.abs(a[h]))
    for h in range(g):
        at = rows == h
        N = int(at.sum())
        if N:
            w = abs(float(s[h]))
            eda[h] = eu[at].T @ np.abs(x[at]) + (row_split + (N + 40) * E) * ((u[at] + eu[at]).T @ np.abs(x[at]))
            edb[h] = w * (row_split + (N + 40) * E) * (np.abs(dout[at]).T @ np.abs(v[at]))
    if need_dx:
        if dbase is not None:
            edx += E * np.abs(dbase)
        within(val(got[0]), dx, edx + half(dtype) * 1.01 * (np.abs(dx) + edx), "dx")
    else:
        assert got[0] is None
    within(val(got[1]), da, eda + half(gdtype) * 1.01 * (np.abs(da) + eda), "da")
    within(val(got[2]), db, edb + half(gdtype) * 1.01 * (np.abs(db) + edb), "db")


def grad_inputs(seed, m, k, n, r, g, dtype, x8):
    rng, x, a, b, s = make(seed, m, k, n, r, g, dtype)
    xs = None
    xv = val(x)
    if x8:
        x, xs = G.mxfp8_quantize(x)
        xv = oracle.mxfp8_values(x.view(torch.uint8).cpu().numpy(), xs.cpu().numpy())
    v = rand(rng, (m, r), F32)
    return rng, x, xs, xv, a, b, s, v, rand(rng, (m, n), dtype), rand(rng, (m, k), dtype)


@pytest.mark.parametrize("types", [(BF, F32, False), (BF, BF, False), (BF, F32, True), (BF, BF, True), (F32, F32, False), (F32, BF, False)])
@pytest.mark.parametrize("case", range(len(GRADS)))
def test_gradients(case, types):
    m, k, n, r, sizes = GRADS[case]
    dtype, gdtype, x8 = types
    say("grad", GRADS[case][:4], types)
    g = len(sizes)
    rng, x, xs, xv, a, b, s, v, dout, dbase = grad_inputs(case, m, k, n, r, g, dtype, x8)
    rows = oracle.row_groups(sizes, m)
    (dx, c1), (da, c2), (db, c3) = framed((m, k), dtype), framed((g, r, k), gdtype), framed((g, n, r), gdtype)
    ws = torch.empty(G.workspace_bytes("lora_grad", m, k, n, g, r, dtype), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)                                        # NaN wherever it is read before it is written
    got = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes), dbase=dbase, scaling=s, x_scale=xs, out=(dx, da, db), workspace=ws)
    c1(), c2(), c3()
    check_grads(got, xv, val(v), val(dout), val(a), val(b), rows, val(s), val(dbase), dtype, gdtype)
    none = torch.from_numpy(rows < 0).to(DEV)
    assert torch.equal(dx[none], dbase[none])
    if m and k and n:
        assert G.read_device_status(ws) == (1 if min(sizes) < 0 else 0) | (2 if sum(max(z, 0) for z in sizes) > m else 0)
    # in place, and without dx: the same
    inplace = dbase.clone()
    got = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes), dbase=inplace, scaling=s, x_scale=xs, out=(inplace, None, None), grad_dtype=gdtype)
    assert torch.equal(inplace, dx) and torch.equal(got[1], da) and torch.equal(got[2], db)
    got = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes), scaling=s, x_scale=xs, need_dx=False, grad_dtype=gdtype)
    assert got[0] is None and torch.equal(got[1], da) and torch.equal(got[2], db)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_without_base_and_scaling(dtype):
    say("grad plain", dtype)
    m, k, n, r, sizes = 90, 130, 77, 10, [40, 0, 45]
    rng, x, xs, xv, a, b, s, v, dout, _ = grad_inputs(31, m, k, n, r, 3, dtype, False)
    got = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes))
    rows = oracle.row_groups(sizes, m)
    check_grads(got, xv, val(v), val(dout), val(a), val(b), rows, np.ones(3), None, dtype, F32)
    assert not bool(got[0][85:].any())


@pytest.mark.parametrize("x8", [False, True])
def test_gradients_and_values_behind_the_groups(x8):
    """NaN in rows past the last group, and a NaN adapter without rows, reach nothing."""
    say("grad NaN", x8)
    m, k, n, r, sizes = 100, 192, 136, 16, [40, 0, 33]
    rng, x, xs, xv, a, b, s, v, dout, dbase = grad_inputs(32, m, k, n, r, 3, BF, x8)
    args = dict(dbase=dbase, scaling=s, x_scale=xs)
    good = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes), **args)
    if x8:
        xs[73:] = 255
    else:
        x[73:] = float("nan")
    v[73:], dout[73:], a[1], b[1], s[1] = float("nan"), float("inf"), float("nan"), float("nan"), float("nan")
    got = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes), **args)
    assert all(torch.equal(p, q) for p, q in zip(good, got))


@pytest.mark.parametrize("wide", [1, 16])
@pytest.mark.parametrize("types", [(BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("knr", [(131, 77, 11), (75, 264, 24), (192, 136, 40), (515, 131, 100)])
def test_gradients_of_non_finite_neighbours_at_odd_sizes(knr, types, wide):
    """NaN in everything of one group, and behind the last, reaches no other group, also where a group ends inside a tile."""
    say("grad non-finite odd", knr, types, wide)
    dtype, x8 = types
    k, n, r = knr[0] // 32 * 32 if x8 else knr[0], knr[1], knr[2]
    sizes, m = [33 * wide, 21 * wide, 40 * wide], 101 * wide
    rng, x, xs, xv, a, b, s, v, dout, dbase = grad_inputs(34, m, k, n, r, 3, dtype, x8)
    args = dict(dbase=dbase, scaling=s, x_scale=xs)
    good = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes), **args)
    for at in (slice(33 * wide, 54 * wide), slice(94 * wide, m)):
        if x8:
            xs[at] = 255
        else:
            x[at] = float("nan")
        v[at], dout[at] = float("inf"), float("nan")
    a[1], b[1] = float("inf"), float("nan")
    got = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes), **args)
    keep = torch.ones(m, dtype=torch.bool, device=DEV)
    keep[33 * wide:54 * wide] = False
    assert torch.equal(got[0][keep], good[0][keep]) and bool(got[0][~keep].isnan().all())
    for p, q in zip(got[1:], good[1:]):
        assert torch.equal(p[[0, 2]], q[[0, 2]]) and not bool(p[1].isfinite().any())


def test_gradients_against_differences():
    """The loss sum(w * ragged_lora(x, a, b)) in fp32 against central differences of the call itself; the call is linear in
    x, in a and in b, so the quotient is exact but for rounding: 2^-24 of a loss of m n terms over the step."""
    say("differences")
    m, k, n, r, sizes = 24, 32, 40, 4, [10, 0, 12]
    rng, x, a, b, s = make(33, m, k, n, r, 3, F32)
    w = rand(rng, (m, n), F32)
    v = torch.empty(m, r, device=DEV)
    gs = ints(sizes)
    G.ragged_lora(x, a, b, gs, scaling=s, v=v)
    dx, da, db = G.ragged_lora_grad(x, v, w, a, b, gs, scaling=s)

    def loss():
        return float((G.ragged_lora(x, a, b, gs, scaling=s).double() * w.double()).sum())

    for leaf, grad in ((x, dx), (a, da), (b, db)):
        for _ in range(6):
            i = tuple(int(rng.integers(0, d)) for d in leaf.shape)
            old = leaf[i].clone()
            leaf[i] = old + 0.5
            up = loss()
            leaf[i] = old - 0.5
            down = loss()
            leaf[i] = old
            assert abs((up - down) - float(grad[i])) <= 60 * E * m * n + 1e-5 * abs(float(grad[i]))


# ---------------------------------------------------------------------------------------------------------------
# as they are used: beside the projections, captured, on other streams


def test_step_of_a_layer_with_adapters():
    """Tokens sorted by expert, the experts' projection, their adapters, and the backward pass with the input in 8 bits."""
    say("layer")
    tokens, top_k, k, n, r, g = 50, 2, 96, 128, 8, 4
    rng, x, a, b, s = make(40, tokens, k, n, r, g, BF)
    w = rand(rng, (g, k, n), BF, k ** -0.5)
    experts = ints(np.stack([rng.permutation(g)[:top_k] for _ in range(tokens)]).tolist())
    sx, _, gs, s2c, c2s = G.moe_permute(x, experts, g)
    y = G.ragged_dot_m(sx, w, gs)
    v = torch.empty(tokens * top_k, r, device=DEV)
    before = y.clone()
    G.ragged_lora(sx, a, b, gs, base=y, out=y, scaling=s, v=v)
    rows = oracle.row_groups(gs.cpu().numpy(), tokens * top_k)
    want, _ = oracle.ragged_lora(val(sx), val(a), val(b), rows, val(s), val(before))
    _, eo = bounds(val(sx), val(a), val(b), rows, val(s), BF, True, want, val(before))
    within(val(y), want, eo)
    dy = rand(rng, (tokens * top_k, n), BF)
    c8, s8 = G.mxfp8_quantize(sx)
    dsx = G.ragged_dot_m(dy, w, gs, rhs_layout="nk")
    base = val(dsx)
    dsx, da, db = G.ragged_lora_grad(c8, v, dy, a, b, gs, dbase=dsx, scaling=s, x_scale=s8, out=(dsx, None, None))
    xv = oracle.mxfp8_values(c8.view(torch.uint8).cpu().numpy(), s8.cpu().numpy())
    check_grads((dsx, da, db), xv, val(v), val(dy), val(a), val(b), rows, val(s), base, BF, F32)
    # rows in their own order give what the sorted ones do
    copies = x[torch.arange(tokens * top_k, device=DEV) // top_k]
    base = before[c2s.long()]
    other = G.ragged_lora(copies, a, b, row_group=experts.reshape(-1), base=base, scaling=s)
    want, _ = oracle.ragged_lora(val(copies), val(a), val(b), experts.reshape(-1).cpu().numpy(), val(s), val(base))
    _, eo = bounds(val(copies), val(a), val(b), experts.reshape(-1).cpu().numpy(), val(s), BF, True, want, val(base))
    within(val(other), want, eo)


def test_captured_and_replayed_with_eager_calls_between():
    say("graph")
    m, k, n, r, g = 64, 512, 264, 16, 6
    rng, x, a, b, s = make(41, m, k, n, r, g, BF)
    base, dout = rand(rng, (m, n), BF), rand(rng, (m, n), BF)
    gs, rows = ints([10, 20, 0, 4, 20, 5]), ints(rng.integers(-1, g, m))
    v = torch.empty(m, r, device=DEV)

    def step():
        one = G.ragged_lora(x, a, b, row_group=rows, base=base, scaling=s)
        two = G.ragged_lora(x, a, b, gs, base=base, scaling=s, v=v)
        return (one, two, v.clone()) + G.ragged_lora_grad(x, v, dout, a, b, gs, scaling=s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.copy_(rand(rng, (m, k), BF)), dout.copy_(rand(rng, (m, n), BF)), rows.copy_(ints(rng.integers(-1, g, m)))
        gs.copy_(ints(rng.multinomial(m - i, np.full(g, 1 / g)).tolist()))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(p, q) for p, q in zip(kept, step()))


def test_two_streams_at_once():
    say("streams")
    m, k, n, r, g = 300, 1024, 512, 16, 4
    rng, x, a, b, s = make(42, m, k, n, r, g, BF)
    gs, dout = ints([100, 50, 0, 149]), rand(rng, (m, n), BF)
    v = torch.empty(m, r, device=DEV)
    want = G.ragged_lora(x, a, b, gs, scaling=s, v=v)
    wg = G.ragged_lora_grad(x, v, dout, a, b, gs, scaling=s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[] for _ in streams]
    for _ in range(10):
        for st, to in zip(streams, got):
            with torch.cuda.stream(st):
                to.append((G.ragged_lora(x, a, b, gs, scaling=s),) + G.ragged_lora_grad(x, v, dout, a, b, gs, scaling=s))
    torch.cuda.synchronize()
    for to in got:
        for res in to:
            assert torch.equal(res[0], want) and all(torch.equal(p, q) for p, q in zip(res[1:], wg))


def test_past_32_bits():
    """x, base and out of more than 2^32 bytes and out of more than 2^31 elements: the last rows."""
    say("long")
    m, k, n, r, g = 66000, 64, 33000, 4, 2
    rng = np.random.default_rng(43)
    a, b = rand(rng, (g, r, k), BF, 0.1), rand(rng, (g, n, r), BF)
    x = torch.zeros(m, k, dtype=BF, device=DEV)
    tail = rand(rng, (5, k), BF)
    x[-5:] = tail
    base = torch.ones(m, n, dtype=BF, device=DEV)
    sizes = [m - 3, 2]
    rows = np.array([0, 0, 1, 1, -1])
    want, _ = oracle.ragged_lora(val(tail), val(a), val(b), rows, None, np.ones((5, n)))
    _, eo = bounds(val(tail), val(a), val(b), rows, None, BF, True, want, np.ones((5, n)))
    full = torch.zeros(m, dtype=torch.int32, device=DEV)
    full[-5:] = ints(rows)
    for pick in (dict(group_sizes=ints(sizes)), dict(row_group=full)):
        out = G.ragged_lora(x, a, b, base=base, **pick)
        within(val(out[-5:]), want, eo)
        assert bool((out[:1000] == 1).all()) and bool((out[-1000:-5] == 1).all())
        del out
    v = torch.ones(m, r, device=DEV)
    dout = base
    dout[:-5] = 0
    got = G.ragged_lora_grad(x, v, dout, a, b, ints(sizes))
    check_grads((got[0][-5:],) + got[1:], val(tail), np.ones((5, r)), np.ones((5, n)), val(a), val(b), rows, np.ones(2), None, BF, F32)
