"""moe_unpermute where every row stays in its place (one copy a token, already in order) and the output is the
input's own array: the rows are weighted in place, whatever their width and alignment."""
import numpy as np
import pytest
import torch

from group_gemm_amd import _binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [7, 9, 15, 64, 515, 519, 1030, 1031, 2056, 7165])   # last pieces of one to seven elements, in a wave's first round and later
def test_rows_weighted_in_place(n, dtype):
    print("[case] in place", n, dtype, flush=True)
    tokens = 301
    r = np.random.default_rng(n)
    y = torch.from_numpy(r.standard_normal((tokens, n)).astype(np.float32)).to(DEV).to(dtype)
    w = torch.from_numpy((r.random((tokens, 1)) + 1).astype(np.float32)).to(DEV)
    i = torch.arange(tokens, dtype=torch.int32, device=DEV)
    want = (y.double() * w.double()).to(torch.float32).to(dtype)   # one fp32 product, then one rounding
    apart = B.moe_unpermute(y, i, w, out_dtype=dtype)
    assert torch.equal(apart, want)
    B.moe_unpermute(y, i, w, out=y)
    assert torch.equal(y, want)
