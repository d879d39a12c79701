"""The scale panels from row-major scales (CPU): the line that README.md gives for weights that exist already."""
import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("g,n,k", [(2, 5, 32), (3, 4, 256), (1, 7, 288), (2, 3, 2880)])
def test_row_major_scales_to_panels(g, n, k):
    scale = np.random.default_rng(k).integers(0, 256, (g, n, k // 32)).astype(np.uint8)
    s = torch.from_numpy(scale)
    panels = torch.nn.functional.pad(s, (0, -s.shape[-1] % 8)).unflatten(-1, (-1, 8)).movedim(-3, -2).contiguous()
    assert panels.shape == (g, -(-k // 256), n, 8)
    assert np.array_equal(panels.numpy(), oracle.mxfp4_panels(scale))
    rows = s[0]
    panels = torch.nn.functional.pad(rows, (0, -rows.shape[-1] % 8)).unflatten(-1, (-1, 8)).movedim(-3, -2).contiguous()
    assert np.array_equal(panels.numpy(), oracle.mxfp4_panels(scale[0]))
