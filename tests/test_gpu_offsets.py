"""Offsets out of order in the appends to both paged caches and in the 4-bit
cache's read: reported however far they drop (blocks look for their request by
its offset, and may pass over the wrong one)."""
import numpy as np
import pytest

from tests.block_util import BlockBatch
from tests.decode_util import Batch
from tests.test_gpu_block_kv import run_append as block_append
from tests.test_gpu_block_kv import run_read as block_read
from tests.test_gpu_paged_kv import run_append as byte_append

pytestmark = pytest.mark.gpu

BOUNDS, T = 6, 62
CU = [[20, 55, 31, 43], [0, 40, 8, 62], [0, 10, 12, 40, 8, 20, 62], [0, 62, 0], [-1, 5, 62], [0, 63, 62], [63, 62],
      [0] * 300 + [40] + [2] * 500 + [62], [0] * 900 + [62, 1, 62]]


def batch(make, cu, **kw):
    """T rows; each request has 70 tokens' room, as far as a request can use it."""
    n = len(cu) - 1
    bt = make([T] + [0] * (n - 1), [70] * n, Hq=1, Hkv=1, D=64, page=128, seed=1, **kw)
    bt.cu = np.array(cu, dtype=np.int32)
    return bt


@pytest.mark.parametrize("cu", CU)
def test_offsets_out_of_order_are_reported(cu):
    assert block_append(batch(BlockBatch, cu))["st"] == BOUNDS
    assert block_read(batch(BlockBatch, cu))[1] == BOUNDS
    if len(cu) < 100:
        assert byte_append(batch(Batch, cu), 0, "half", False)["st"] == BOUNDS


@pytest.mark.parametrize("cu", [[0, 62], [3, 40, 40, 60], [0] * 300 + [40] * 500 + [62]])
def test_offsets_in_order_are_not(cu):
    assert block_append(batch(BlockBatch, cu))["st"] == 0
    assert block_read(batch(BlockBatch, cu))[1] == 0
    if len(cu) < 100:
        assert byte_append(batch(Batch, cu), 0, "half", False)["st"] == 0
