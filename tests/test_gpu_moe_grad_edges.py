"""moe_permute_grad and moe_unpermute_grad where a value is not finite, a copy has no sorted row, or
tensors lie in one another."""
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


def same(got, want):
    """equal, NaN equal to NaN"""
    return np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top_k", [1, 3, 9])
@pytest.mark.parametrize("n", [5, 7, 8, 24, 512, 515, 1030])   # by elements, one wave, two waves; a last piece that overlaps
def test_nonfinite_dout_of_tokens_with_unrouted_copies(n, top_k, dtype):
    """dweights is 0 where a copy has no sorted row, whatever its token's dout holds; elsewhere an infinity or
    a NaN of dout gives what the sum in 64 bits gives.  Whole numbers of at most 4 bits: every finite sum is
    exact (1030 * 64 < 2^24)."""
    say("non-finite dout", n, top_k, dtype)
    tokens = 9
    r = np.random.default_rng(n + top_k)
    e = r.integers(0, 4, (tokens, top_k))
    e[:6, 0] = -1                                    # a copy that was not routed, in every token with such a dout
    e[5] = -1
    _, _, _, s2c, c2s = oracle.moe_permute(np.zeros((tokens, 1), np.float32), e, 4)
    y = r.integers(-8, 9, (tokens * top_k, n)).astype(np.float32)
    y[y == 0] = 1                                    # (an infinity of dout meets no zero in a routed row)
    dout = r.integers(-8, 9, (tokens, n)).astype(np.float32)
    dout[0, 0], dout[1, n - 1], dout[2, n // 2] = np.inf, -np.inf, np.nan
    dout[3, :] = np.nan
    dout[5, n - 1] = np.inf
    dout[6, n - 1], dout[7, 0] = np.nan, np.inf      # tokens whose copies are all routed
    w = r.integers(1, 9, (tokens, top_k)).astype(np.float32)
    dout_d, y_d = dev(dout).to(dtype), dev(y).to(dtype)
    dy, dw = B.moe_unpermute_grad(dout_d, y_d, dev(c2s), dev(s2c), dev(w))
    with np.errstate(invalid="ignore"):
        want_y, want_w, _ = oracle.moe_unpermute_grad(W.to_numpy_raw(dout_d), W.to_numpy_raw(y_d), c2s, s2c, w)
    absent = (c2s < 0).reshape(tokens, top_k)
    assert absent[:6, 0].all() and not want_w[absent].any()
    got = dw.double().cpu().numpy()
    assert not got[absent].any(), "a copy without a sorted row has a weight gradient"
    assert same(got, want_w)
    assert same(dy.double().cpu().numpy(), want_y)   # products of whole numbers of at most 4 bits: exact in bf16


def test_outputs_in_an_input_are_refused():
    """Only where rows are still read is the call refused: beside an input, and weights' own array, stay allowed."""
    say("in place")
    tokens, top_k, n = 6, 2, 16
    M = tokens * top_k
    buf = torch.arange(2 * M * n, device=DEV, dtype=F32).view(2 * M, n)
    d = buf[:M]
    i = torch.arange(M, dtype=torch.int32, device=DEV)
    w = torch.rand(tokens, top_k, device=DEV)
    before = buf.clone()
    for out in (d[:tokens], d[tokens:], buf[M - 1:M + 5]):
        with pytest.raises(ValueError, match="overlaps dsorted"):
            B.moe_permute_grad(d, i, top_k, out=out)
    with pytest.raises(ValueError, match="dweights overlaps y"):
        B.moe_unpermute_grad(d[:tokens].clone(), d, i, i, w, out=(None, d.view(-1)[:M].view(tokens, top_k)))
    wide = torch.rand(M + 1, device=DEV)
    with pytest.raises(ValueError, match="dweights overlaps weights"):
        B.moe_unpermute_grad(d[:tokens].clone(), d, i, i, wide[:M].view(tokens, top_k), out=(None, wide[1:].view(tokens, top_k)))
    assert torch.equal(buf, before)
    want = B.moe_permute_grad(d, i, top_k)
    assert torch.equal(B.moe_permute_grad(d, i, top_k, out=buf[M:M + tokens]), want) and torch.equal(d, before[:M])


@pytest.mark.parametrize("top_k", [2, 19])
@pytest.mark.parametrize("n", [24, 1030])
def test_weight_gradients_into_the_weights(n, top_k):
    say("dweights over weights", n, top_k)
    tokens = 21
    r = np.random.default_rng(n + top_k)
    e = r.integers(-1, 5, (tokens, top_k))
    _, _, _, s2c, c2s = oracle.moe_permute(np.zeros((tokens, 1), np.float32), e, 5)
    dout, y = (dev(r.standard_normal((m, n)).astype(np.float32)) for m in (tokens, tokens * top_k))
    w = dev(r.random((tokens, top_k)).astype(np.float32))
    want = B.moe_unpermute_grad(dout, y, dev(c2s), dev(s2c), w)
    got = B.moe_unpermute_grad(dout, y, dev(c2s), dev(s2c), w, out=(None, w))
    assert got[1].data_ptr() == w.data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
