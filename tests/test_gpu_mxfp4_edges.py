"""MXFP4 at the ends of the number range and at unaligned rows: subnormal values, products whose sums are subnormal
or overflow, and the sort by expert of rows that begin at any byte."""
import numpy as np
import pytest
import torch

import oracle
from group_gemm_amd import _binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print("[case]", *a, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_subnormal_values_are_quantised(dtype):
    """Blocks whose largest magnitude is subnormal have scale 2^-127, and their codes are rounded as any other's."""
    say("subnormals", dtype)
    r = np.random.default_rng(30)
    rows, k, least = 64, 256, -133 if dtype == BF else -149
    v = r.integers(-255, 256, (rows, k)) / 128 * 2.0 ** r.integers(least, -118, (rows, k))
    v[:8] = r.integers(-255, 256, (8, k)) * 2.0 ** -134
    v[8], v[9] = 2.0 ** -127, -1.5 * 2.0 ** -127
    x = torch.from_numpy(v).to(dtype).to(DEV)
    want_c, want_s = oracle.mxfp4_quantize(x.double().cpu().numpy())
    assert want_s.min() == 0 and (want_c[8] == 0x22).all() and (want_c[9] == 0xBB).all()   # 1 and -1.5 times 2^-127
    c, s = B.mxfp4_quantize(x)
    assert np.array_equal(raw(s), oracle.mxfp4_panels(want_s)) and np.array_equal(raw(c), want_c)
    c, s = B.mxfp4_quantize_weights(x.view(1, rows, k).transpose(1, 2).contiguous())
    assert np.array_equal(raw(s)[0], oracle.mxfp4_panels(want_s)) and np.array_equal(raw(c)[0], want_c)


@pytest.mark.parametrize("m,n,kernel", [(3, 64, 0), (100, 264, 1), (1700, 5000, 2)])
def test_products_at_the_ends_of_the_range(m, n, kernel):
    """Scales at both ends: results that are subnormal in fp32 are kept, those past its range are infinite."""
    say("range", m, n)
    g, k = 2, 768
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert B.lib().gg_mxfp4_kernel(m, k, n, g, cus) == kernel
    gen = torch.Generator(device=DEV).manual_seed(m)
    x = torch.randint(0, 256, (m, k // 2), dtype=torch.uint8, device=DEV, generator=gen)
    w = torch.randint(0, 256, (g, n, k // 2), dtype=torch.uint8, device=DEV, generator=gen)
    gs = dev(np.array([m // 2, m - m // 2], np.int32))
    rows, cols = slice(0, min(m // 2, 8)), slice(0, 64)      # of the first group
    for a, b in ((127, 127), (60, 60), (50, 60), (0, 127), (127, 0), (200, 150), (254, 150)):
        xs, ws = torch.full((3, m, 8), a, dtype=torch.uint8, device=DEV), torch.full((g, 3, n, 8), b, dtype=torch.uint8, device=DEV)
        out = B.ragged_dot_m_mxfp4(x, w, gs, xs, ws, out_dtype=F32)[rows, cols].double().cpu().numpy()
        av, bv = oracle.mxfp4_values(raw(x[rows]), raw(xs[:, rows])), oracle.mxfp4_values(raw(w[0, cols]), raw(ws[0][:, cols]))
        want, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
        big = np.finfo(np.float32).max
        if a == 254:
            assert (mag > big).all() and not np.isfinite(out).any()
        else:   # (2^-149: the spacing of the subnormals)
            assert mag.max() < big and (np.abs(out - want) <= (k / 8 + 32) * (2.0 ** -23 * mag + 2.0 ** -149)).all(), (a, b)
            assert (out != 0).any()


@pytest.mark.parametrize("shift", [0, 1, 8])
def test_permute_of_rows_at_any_byte(shift):
    say("permute, rows at byte", shift)
    r = np.random.default_rng(31)
    tokens, top_k, k, g = 57, 3, 544, 6
    codes, scale = oracle.mxfp4_quantize(r.standard_normal((tokens, k)))
    experts = r.integers(-1, g, (tokens, top_k)).astype(np.int32)
    M, n = tokens * top_k, k // 2

    def at(rows):
        b = torch.full((rows * n + 64,), 0xAB, dtype=torch.uint8, device=DEV)
        return b, b[shift:shift + rows * n].view(rows, n)
    _, x = at(tokens)
    x.copy_(dev(codes))
    buf, sx = at(M)
    out = (sx.view(B.FP4), None, None, None, None)
    _, ss, gs, s2c, c2s = B.moe_permute(x.view(B.FP4), dev(experts), g, x_scale=dev(oracle.mxfp4_panels(scale)), out=out)
    ox, os_, ogs, os2c, oc2s = oracle.moe_permute(codes, experts, g, scale)
    assert np.array_equal(raw(sx), ox) and np.array_equal(raw(ss), oracle.mxfp4_panels(os_))
    assert np.array_equal(gs.cpu().numpy(), ogs) and np.array_equal(s2c.cpu().numpy(), os2c) and np.array_equal(c2s.cpu().numpy(), oc2s)
    assert (buf[:shift] == 0xAB).all() and (buf[shift + M * n:] == 0xAB).all()
