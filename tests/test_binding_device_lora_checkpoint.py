"""The adapters' and the 8-bit checkpoints' calls run on their tensors' device, whichever is current (CPU: stand-ins for the
library and torch's device functions, from test_binding_device.py)."""
import pytest
import torch

from group_gemm_amd import _binding as B
from test_binding_device import gpu1, z, GS, U8, I32   # noqa: F401

F = torch.float32
A, BW = (2, 4, 64), (2, 16, 4)
CALLS = {
    "mxfp8_quantize": lambda: B.mxfp8_quantize(z(8, 64)),
    "mxfp8_dequantize": lambda: B.mxfp8_dequantize(z(8, 64, dtype=U8), z(8, 2, dtype=U8)),
    "gated_act_mxfp8": lambda: B.gated_act_mxfp8(z(8, 64), z(8, 64)),
    "gated_act_mxfp8_grad": lambda: B.gated_act_mxfp8_grad(z(8, 64), z(8, 128, dtype=U8), z(8, 4, dtype=U8)),
    "ragged_dot_k_mxfp8": lambda: B.ragged_dot_k(z(8, 64, dtype=U8), z(8, 16), GS, lhs_scale=z(8, 2, dtype=U8)),
    "ragged_lora": lambda: B.ragged_lora(z(8, 64), z(*A), z(*BW), GS, base=z(8, 16)),
    "ragged_lora_grad": lambda: B.ragged_lora_grad(z(8, 64), z(8, 4, dtype=F), z(8, 16), z(*A), z(*BW), GS),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_calls_run_on_their_tensors_device(gpu1, name):   # noqa: F811
    CALLS[name]()
    assert gpu1.calls == [(name, 1, 1001)]
