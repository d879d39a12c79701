"""The fp64 oracle of the adapters and of the 8-bit checkpoints against other ways to compute the same (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from group_gemm_amd import workloads as W


def test_e4m3_values_are_torchs():
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    got = oracle.mxfp8_values(np.tile(c, (1, 1)), np.full((1, 8), 127, np.uint8))[0]
    assert np.array_equal(got, want, equal_nan=True)


def test_quantize_against_torchs_rounding():
    r = np.random.default_rng(1)
    x = (r.standard_normal((64, 128)) * np.exp2(r.integers(-130, 100, (64, 1)))).astype(np.float32)
    codes, scale = oracle.mxfp8_quantize(x)
    b = torch.from_numpy(x.astype(np.float64)).reshape(64, 4, 32)
    q = b / 2.0 ** (torch.from_numpy(scale.astype(np.float64))[..., None] - 127)
    assert float(q.abs().max()) <= 448
    want = q.float().to(torch.float8_e4m3fn).view(torch.uint8).reshape(64, 128)   # x / 2^e is a float again
    assert np.array_equal(want.numpy(), codes)
    # the smallest such power of two: with the next smaller one, the largest value passes 448
    assert bool(((q.abs().amax(-1) > 224) | (torch.from_numpy(scale) == 0)).all())


def test_quantize_differs_from_the_clipping_rule_only_where_that_clips():
    r = np.random.default_rng(2)
    x = r.standard_normal((50, 64)).astype(np.float32)
    codes, scale = oracle.mxfp8_quantize(x)
    c2, s2 = W.mx_quantize(torch.from_numpy(x), 1)
    over = np.abs(x.reshape(50, 2, 32)).max(-1) > 448 * np.exp2(s2.numpy().astype(np.float64) - 127)
    assert over.any() and not over.all()
    assert np.array_equal(scale, s2.numpy() + over)
    same = np.repeat(~over, 32, axis=1)
    assert np.array_equal(codes[same], c2.numpy()[same])
    # and where it clips, a value is more than a rounding (2^-4) off
    err = lambda c, s: np.abs(oracle.mxfp8_values(c, s) - x)[~same]
    assert (err(codes, scale) <= 2.0 ** -4 * np.abs(x[~same]) + 2.0 ** -9).all()
    assert not (err(c2.numpy(), s2.numpy()) <= 2.0 ** -4 * np.abs(x[~same]) + 2.0 ** -9).all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gate_slope_is_the_difference_quotient(act):
    x = np.linspace(-12, 12, 4001)
    f, d = oracle.gate_and_slope(x, act)
    step = 1e-5
    q = (oracle.gate_and_slope(x + step, act)[0] - oracle.gate_and_slope(x - step, act)[0]) / (2 * step)
    assert np.abs(q - d).max() < 1e-8          # step^2 / 6 times the third derivative, and 1e-15 / step
    tf = torch.nn.functional.silu if act == "silu" else lambda t: torch.nn.functional.gelu(t, approximate="tanh")
    assert np.abs(tf(torch.from_numpy(x)).numpy() - f).max() < 1e-14


def test_lora_against_dense_weights_and_autograd():
    r = np.random.default_rng(4)
    m, k, n, rank, g = 13, 7, 9, 3, 4
    x, a, b = r.standard_normal((m, k)), r.standard_normal((g, rank, k)), r.standard_normal((g, n, rank))
    base, dout, s = r.standard_normal((m, n)), r.standard_normal((m, n)), r.standard_normal(g)
    rows = oracle.row_groups([3, 0, 5, 2], m)
    out, v = oracle.ragged_lora(x, a, b, rows, s, base)
    tx, ta, tb = (torch.from_numpy(t).requires_grad_() for t in (x, a, b))
    dense = torch.cat([(torch.from_numpy(s)[:, None, None] * tb @ ta), torch.zeros(1, n, k, dtype=torch.float64)])
    want = torch.from_numpy(base) + (dense[torch.from_numpy(rows)] @ tx[..., None])[..., 0]
    assert np.allclose(want.detach().numpy(), out, rtol=0, atol=1e-12)
    want.backward(torch.from_numpy(dout))
    for got, leaf in zip(oracle.ragged_lora_grad(x, v, dout, a, b, rows, s), (tx, ta, tb)):
        assert np.allclose(got, leaf.grad.numpy(), rtol=0, atol=1e-12)


def test_row_groups_clamps():
    assert oracle.row_groups([2, -3, 1], 5).tolist() == [0, 0, 2, -1, -1]
    assert oracle.row_groups([2, 9], 4).tolist() == [0, 0, 1, 1]
