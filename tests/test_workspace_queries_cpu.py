"""Workspace queries of the block-scaled products: 0 for sizes that the calls refuse, whatever their arithmetic would
make of them."""
import pytest

import vocabulary_cross_entropy_row_amd as lce

QUERIES = ["lce_linear_blocks_workspace_bytes", "lce_linear_blocks_forward_workspace_bytes", "lce_linear_blocks_backward_workspace_bytes"]
TOP = (1 << 63) - 1


@pytest.mark.parametrize("name", QUERIES)
@pytest.mark.parametrize("sizes", [(TOP, 128, 128), (1, TOP, 1), (128, 128, TOP), (1 << 62,) * 3, (1 << 23, 128, 128), (128, 128, 1 << 23),
                                   (128, 1 << 24, 128), (-1, 128, 128), (1, 0, 1), (1, 1, 0)])
def test_refused_sizes(name, sizes):
    assert getattr(lce.lib(), name)(*sizes) == 0


def up(v, unit):
    return -(-v // unit) * unit


@pytest.mark.parametrize("n,K,M", [(64, 8192, 256), (4096, 8192, 8192), (0, 300, 500), (517, 1001, 2051)])
def test_others(n, K, M):
    """The quantised operands with their scales, each on 256 bytes, and what the products take to add up their splits."""
    product, forward, backward = (getattr(lce.lib(), name) for name in QUERIES)
    rows, blocks = up(K, 16), up(K, 128) // 128
    assert forward(n, K, M) == (up(n * rows, 256) + up(n * blocks, 256) + up(M * rows, 256) + up(up(M, 128) // 128 * blocks, 256)
                                + up(product(n, K, M), 256))
    of_m, of_n = up(M, 128) // 128, up(n, 128) // 128
    assert backward(n, K, M) == (up(n * up(M, 16), 256) + up(M * up(n, 16), 256) + up(n * of_m, 256) + up(M * of_n, 256)
                                 + up(4 * of_n * M, 256) + up(max(product(n, M, K), product(M, n, K)), 256))
