"""Every call of the binding runs on its tensors' device, whichever is current (CPU: the library and torch's device
functions are stand-ins, so nothing is launched).  With the current device left as it is, a call on another GPU's
tensors would launch on the current GPU, as the default stream's handle is the same on both."""
import contextlib
import types

import pytest
import torch

from group_gemm_amd import _binding as B

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


class Library:
    """Records (name, current device, stream) of every launching call; sizes come from the real library."""

    def __init__(self, cuda):
        self.cuda, self.calls, self.real = cuda, [], B.lib()

    def __getattr__(self, name):
        if name == "gg_workspace_bytes":
            return self.real.gg_workspace_bytes

        def call(*args):
            self.calls.append((name, self.cuda.current, args[-1]))
            return 0
        return call


@pytest.fixture
def gpu1(monkeypatch):
    """CPU tensors that the binding takes for tensors of cuda:1, while cuda:0 is current."""
    cuda = types.SimpleNamespace(current=0)

    @contextlib.contextmanager
    def device(dev):
        before, cuda.current = cuda.current, dev.index
        yield
        cuda.current = before

    lib = Library(cuda)
    real_call = B._call
    dev = torch.device("cuda", 1)
    monkeypatch.setattr(B, "_tensor", lambda *a, **k: None)
    monkeypatch.setattr(B, "_call", lambda name, d, *args: real_call(name, dev, *args))
    monkeypatch.setattr(B, "_lib", lib)
    monkeypatch.setattr(B, "lib", lambda: lib)
    monkeypatch.setattr(B, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: cuda.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=-1))
    yield lib
    assert cuda.current == 0


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def fp4(*shape):
    return z(*shape, dtype=U8).view(B.FP4)


GS = torch.tensor([4, 4], dtype=I32)
I16 = torch.arange(16, dtype=I32)
CALLS = {
    "ragged_dot_m": lambda: B.ragged_dot_m(z(8, 64), z(2, 64, 16), GS),
    "ragged_dot_m_nk": lambda: B.ragged_dot_m(z(8, 64), z(2, 16, 64), GS, rhs_layout="nk"),
    "ragged_dot_m_epilogue": lambda: B.ragged_dot_m(z(8, 64), z(2, 64, 16), GS, alpha=2.0),
    "ragged_dot_m_noalloc": lambda: B.ragged_dot_m_noalloc(z(8, 64), z(2, 64, 16), GS, out=z(8, 16)),
    "ragged_dot_m_gated": lambda: B.ragged_dot_m_gated(z(8, 64), z(2, 64, 16), z(2, 64, 16), GS),
    "ragged_dot_k": lambda: B.ragged_dot_k(z(8, 64), z(8, 16), GS),
    "ragged_dot_k_epilogue": lambda: B.ragged_dot_k(z(8, 64), z(8, 16), GS, alpha=2.0),
    "padded_dot": lambda: B.padded_dot("m", z(8, 64), z(2, 64, 16), GS, 4),
    "moe_permute": lambda: B.moe_permute(fp4(8, 32), z(8, 2, dtype=I32), 4, x_scale=z(1, 8, 8, dtype=U8)),
    "moe_unpermute": lambda: B.moe_unpermute(z(16, 8), I16, torch.ones(8, 2)),
    "moe_permute_grad": lambda: B.moe_permute_grad(z(16, 8), I16, 2),
    "moe_unpermute_grad": lambda: B.moe_unpermute_grad(z(8, 8), z(16, 8), I16, I16, torch.ones(8, 2)),
    "mxfp4_quantize": lambda: B.mxfp4_quantize(z(8, 64)),
    "mxfp4_quantize_weights": lambda: B.mxfp4_quantize_weights(z(2, 64, 16)),
    "mxfp4_dequantize": lambda: B.mxfp4_dequantize(fp4(8, 32), z(1, 8, 8, dtype=U8)),
    "ragged_dot_m_mxfp4": lambda: B.ragged_dot_m_mxfp4(fp4(8, 32), fp4(2, 16, 32), GS, z(1, 8, 8, dtype=U8), z(2, 1, 16, 8, dtype=U8)),
    "gg_schedule": lambda: B.build_schedule(GS, 8, 16, 4, 16),
    "gg_read_device_status": lambda: B.read_device_status(z(256, dtype=U8)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_calls_run_on_their_tensors_device(gpu1, name):
    CALLS[name]()
    assert gpu1.calls == [(name, 1, 1001)]


def test_a_failing_call_names_itself(gpu1, monkeypatch):
    monkeypatch.setattr(gpu1, "mxfp4_quantize", lambda *a: 4, raising=False)
    monkeypatch.setattr(gpu1, "gg_status_string", lambda code: b"misaligned pointer", raising=False)
    with pytest.raises(B.GGError, match="mxfp4_quantize"):
        B.mxfp4_quantize(z(8, 64))
