"""Which kernel the MXFP4 product takes (CPU): the GPU tests' shapes for long groups, and the rule's edges, on 256
compute units."""
import pytest

import test_gpu_mxfp4
import test_gpu_mxfp4_tile
from group_gemm_amd import _binding as B

STREAM, BLOCK, TILE = 0, 1, 2


def kernel(m, k, n, g, cus=256):
    return B.lib().gg_mxfp4_kernel(m, k, n, g, cus)


@pytest.mark.parametrize("case", test_gpu_mxfp4_tile.CASES)
def test_shapes_of_the_long_groups_tests(case):
    assert kernel(*test_gpu_mxfp4_tile.shape(case)) == TILE


def test_shapes_of_the_other_product_tests():
    """Each of the three kernels has several of the general test's shapes."""
    taken = [kernel(m, k, n, len(gs)) for m, k, n, gs, *_ in test_gpu_mxfp4.CASES + test_gpu_mxfp4.TILES + test_gpu_mxfp4.LONG]
    assert min(taken.count(STREAM), taken.count(BLOCK), taken.count(TILE)) >= 3
    assert all(kernel(m, k, n, len(gs)) == TILE for m, k, n, gs, _ in test_gpu_mxfp4.LONG)


def test_edges():
    assert kernel(4 * 128, 2880, 5760, 128) == STREAM and kernel(5 * 128, 2880, 5760, 128) == BLOCK   # rows a group
    assert kernel(64, 3328, 512, 16) == STREAM and kernel(64, 3360, 512, 16) == BLOCK                 # a tile's rows in LDS
    assert kernel(8, 6144, 512, 2) == STREAM and kernel(8, 6176, 512, 2) == BLOCK                     # half a tile's
    assert kernel(8192, 544, 14336, 8) == TILE and kernel(8192, 512, 14336, 8) == BLOCK               # at least three panels
    assert kernel(8192, 4096, 14336, 8) == TILE and kernel(1500, 2880, 1447, 32) == BLOCK
    for m, k, n in ((0, 64, 8), (4, 0, 8), (0, 0, 0)):
        assert kernel(m, k, n, 2) in (STREAM, BLOCK)
    assert kernel(0, 4096, 8192, 2) in (STREAM, BLOCK)


def test_refused_shapes():
    assert kernel(-1, 64, 8, 2) == kernel(4, 48, 8, 2) == kernel(4, 64, -8, 2) == kernel(4, 64, 8, 0) == kernel(4, 64, 8, 1025) == -1
    assert kernel(4, 64, 8, 2, 0) == kernel(1 << 31, 64, 8, 2) == kernel(4, 1 << 25, 8, 2) == kernel((1 << 31) - 1, 32, 1, 1) == -1
