"""Host checks of the gradients of permute and un-permute (CPU): outputs that lie in an input or in each other.
Every call below fails validation, so no pointer is dereferenced."""
import pytest

from group_gemm_amd import _binding as B

UNSUPPORTED = 6
AT = 0x100000   # arrays of 16 tokens, top_k 2, 8 columns of bf16: rows 512 bytes, tokens 256, per copy 128


@pytest.mark.parametrize("dx", [AT, AT + 510, AT - 254, AT + 256, AT - 510])
def test_permute_grad_in_place(dx):
    out_type = 0 if dx == AT - 510 else 1   # (an fp32 dx of 512 bytes reaches further)
    dx += 2 if out_type == 0 else 0
    assert B.lib().moe_permute_grad(AT, 2 * AT, dx, 16, 2, 8, 1, out_type, None) == UNSUPPORTED


def test_permute_grad_over_the_index():
    assert B.lib().moe_permute_grad(AT, 2 * AT, 2 * AT + 64, 16, 2, 8, 1, 1, None) == UNSUPPORTED


@pytest.mark.parametrize("change", [dict(dy=2 * AT), dict(dy=2 * AT + 510), dict(dy=2 * AT - 510), dict(dy=AT + 254), dict(dy=3 * AT + 124),
                                    dict(dy=4 * AT), dict(dy=5 * AT + 2), dict(dy=7 * AT + 126), dict(dw=AT), dict(dw=2 * AT + 508),
                                    dict(dw=3 * AT), dict(dw=4 * AT - 124), dict(dw=5 * AT + 4), dict(dw=6 * AT + 508)])
def test_unpermute_grad_in_place(change):
    a = dict(dout=AT, y=2 * AT, c=3 * AT, s=4 * AT, w=5 * AT, dy=6 * AT, dw=7 * AT) | change
    assert B.lib().moe_unpermute_grad(a["dout"], a["y"], a["c"], a["s"], a["w"], a["dy"], a["dw"], 16, 2, 8, 1, None) == UNSUPPORTED
