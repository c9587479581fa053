"""Block-scaled products around the size from which large tiles take over, with every kind of remainder."""

import pytest

import test_gpu_ops as ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1280, 4096, 384), (1288, 4096, 384), (1500, 4096, 640), (1536, 4096, 256), (1552, 4096, 128),
                                   (880, 7168, 512), (1024, 6144, 384), (2900, 2048, 256)])
def test_products_at_the_border_of_the_large_tiles(M, N, K):
    ops.test_block_matmul(M, N, K)
