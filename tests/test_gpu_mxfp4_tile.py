"""GPU parity of the MXFP4 product's kernel for long groups, every element against a product in 64 bits, at shapes
that are shown to take it: more groups than one read of the tile table's lanes covers, empty groups at the
table's 16-group borders, groups shorter than half a tile, several tiles a workgroup, both orders of a group's
tiles, whole and element-wise result stores, rows behind the last group, and calls side by side.

The bound is the one of test_gpu_mxfp4.py: exact 4-bit products, fewer than k / 8 + 32 additions of which each
is off by at most 2^-23 of the sum of magnitudes, and half a step, 2^-8 of the value, for a bf16 result.
"""
import numpy as np
import pytest
import torch

from group_gemm_amd import _binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TILE = 2

CASES = [
    # groups, mean rows, k, n, rows behind, type
    (17, 400, 800, 1544, 37, BF),       # one group past the first 16; n whole in bf16 and fp32
    (17, 400, 800, 1544, 0, F32),
    (17, 410, 1056, 1541, 5, BF),       # no row of the result aligned
    (65, 120, 800, 768, 100, BF),       # most row tiles under half full: two of the four waves without rows
    (65, 120, 800, 768, 3, F32),
    (65, 300, 608, 4104, 11, BF),       # over 1100 tiles, several a workgroup; groups shorter than n
    (65, 300, 608, 4099, 0, F32),
    (300, 160, 800, 256, 61, BF),       # groups longer than n: column tiles side by side
    (300, 160, 800, 251, 0, F32),
    (300, 160, 1312, 256, 0, F32),
    (1024, 70, 544, 136, 77, BF),       # the most groups, three panels, the last one part full
    (1024, 72, 768, 132, 0, F32),
]


def say(*a):
    print("[case]", *a, flush=True)


def shape(case):
    g, mean, k, n, tail, _ = case
    return g * mean + tail, k, n, g


def group_sizes(case, r):
    """Sizes with empty groups at the borders of 16, one to three rows in some, some several tiles long, and the
    last group empty or not; their sum is groups x mean."""
    g, mean = case[:2]
    gs = r.integers(1, 2 * mean, g)
    h = np.arange(g)
    gs[r.random(g) < 0.1] = r.integers(1, 4)
    gs[((h % 16 == 0) | (h % 16 == 15)) & (r.random(g) < 0.6)] = 0
    if g > 33:
        gs[32:48] = 0                                  # sixteen empty groups in a row
    if case[4]:
        gs[-1] = 0
    long = g // 2 if g // 2 < 32 or g // 2 >= 48 else 31
    gs[long] = 0
    gs[long] = max(0, g * mean - int(gs.sum()))        # what is left: the longest group
    while gs.sum() > g * mean:
        gs[np.argmax(gs)] -= min(int(gs.sum()) - g * mean, int(gs.max()))
    assert gs.sum() == g * mean and gs.min() >= 0
    return gs.astype(np.int32)


def values(codes, panels):
    """Codes [rows, k/2] and scale panels [ceil(k/256), rows, 8] in 64 bits, by the format."""
    c = codes.to(torch.int64)
    c = torch.stack([c % 16, c // 16], 2).reshape(codes.shape[0], -1)
    e, f = (c % 8) // 2, (c % 2).double()
    v = torch.where(e == 0, f / 2, (1 + f / 2) * torch.exp2((e - 1).double()))
    v = torch.where(c >= 8, -v, v)
    s = panels.permute(1, 0, 2).reshape(codes.shape[0], -1)[:, :v.shape[1] // 32].double()
    return v * torch.exp2(s - 127).repeat_interleave(32, 1)


def operands(case, seed):
    m, k, n, g = shape(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kp = -(-k // 256)

    def codes(*s):
        return torch.randint(0, 256, s, dtype=torch.uint8, device=DEV, generator=gen)

    def scales(*s):   # the bytes past k are NaN: they must not be used
        t = torch.randint(118, 126, s, dtype=torch.uint8, device=DEV, generator=gen)
        if k % 256:
            t[..., -1, :, k % 256 // 32:] = 255
        return t
    return codes(m, k // 2), codes(g, n, k // 2), scales(kp, m, 8), scales(g, kp, n, 8)


def check(out, x, w, xs, ws, gs, k):
    at = 0
    for h, size in enumerate(gs.tolist()):
        if size:
            a, b = values(x[at:at + size], xs[:, at:at + size]), values(w[h], ws[h]).t().contiguous()
            want, mag = a @ b, a.abs() @ b.abs()
            bound = (k / 8 + 32) * 2.0 ** -23 * mag + (2.0 ** -8 * want.abs() if out.dtype == BF else 0)
            off = (out[at:at + size].double() - want).abs()
            assert bool((off <= bound).all()), (h, size, at)   # (a NaN compares false)
        at += size
    assert not out[at:].any(), "rows past the groups are 0"


@pytest.mark.parametrize("case", range(len(CASES)))
def test_tiles(case):
    c = CASES[case]
    say("tile kernel", c)
    m, k, n, g = shape(c)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert B.lib().gg_mxfp4_kernel(m, k, n, g, cus) == TILE
    gs = group_sizes(c, np.random.default_rng(200 + case))
    x, w, xs, ws = operands(c, case)
    lead = 256   # (elements, so that the result begins 16-byte aligned)
    buf = torch.full((m * n + 2 * lead,), float("nan"), dtype=c[5], device=DEV)
    out = buf[lead:lead + m * n].view(m, n)
    status = torch.full((B.workspace_bytes("ragged_m", m, k, n, g, 0, B.FP4),), 0xAB, dtype=torch.uint8, device=DEV)
    B.ragged_dot_m_mxfp4(x, w, torch.from_numpy(gs).to(DEV), xs, ws, out=out, workspace=status)
    check(out, x, w, xs, ws, gs, k)
    assert torch.isnan(torch.cat([buf[:lead], buf[-lead:]])).all(), "wrote outside its output"
    assert B.read_device_status(status) == 0


def test_tiles_side_by_side():
    """Two shapes on two streams, one workspace, then captured and replayed with eager calls in between."""
    say("tile kernel: two streams, graphs")
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    ws, calls, wants = None, [], []
    for i in (2, 4):
        c = CASES[i]
        m, k, n, g = shape(c)
        assert B.lib().gg_mxfp4_kernel(m, k, n, g, cus) == TILE
        if ws is None:
            ws = torch.zeros(B.workspace_bytes("ragged_m", m, k, n, g, 0, B.FP4), dtype=torch.uint8, device=DEV)
        x, w, xs, sc = operands(c, 50 + i)
        gs = torch.from_numpy(group_sizes(c, np.random.default_rng(i))).to(DEV)
        calls.append(lambda x=x, w=w, gs=gs, xs=xs, sc=sc, t=c[5]: B.ragged_dot_m_mxfp4(x, w, gs, xs, sc, out_dtype=t, workspace=ws))
        wants.append(calls[-1]())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(6):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(calls[i]())
    torch.cuda.synchronize()
    assert all(torch.equal(o, wants[i]) for i in range(2) for o in outs[i])
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[i]):
            o = calls[i]()
        graphs.append((graph, o))
    for _ in range(3):
        for i, (graph, o) in enumerate(graphs):
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, wants[i]) and torch.equal(calls[1 - i](), wants[1 - i])
