"""The 8-bit grouped product with the large tiles at K too short to chain them (one tile a workgroup, fewer steps than
the ring has stages, or as many), and at the first K where they are chained.  Inputs, plain form and bounds are those
of many tiles."""
import pytest
import torch

from test_gpu_product_tiles import test_many_tiles as _many_tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


# tiles of 256, 128 and 64 rows
@pytest.mark.parametrize("M,N,G", [(8192, 2304, 4), (8192, 2304, 64), (2048, 2304, 128)])
@pytest.mark.parametrize("K", [1, 128, 250, 384, 512, 520, 640, 641])
@pytest.mark.parametrize("gather", [False, True])
def test_short_products(dev, M, N, G, K, gather):
    _many_tiles(dev, M, N, K, G, 1, gather)
