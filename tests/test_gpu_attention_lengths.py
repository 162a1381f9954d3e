"""Lengths near 2^31 in the attention over both paged caches (include/paged_kv.h,
include/block_kv.h): positions past the page table are reported and not visible,
so such a request gets what any length past the table gives it, and the others
what they get without it, bit for bit."""
import numpy as np
import pytest
import torch

from tests.block_util import BlockBatch
from tests.decode_util import Batch
from tests.test_gpu_block_kv import run_attention as run_blocks
from tests.test_gpu_paged_kv import run_attention as run_bytes

pytestmark = pytest.mark.gpu

BOUNDS, TOP = 6, 2 ** 31 - 1


@pytest.mark.parametrize("make,run", [(Batch, run_bytes), (BlockBatch, run_blocks)])
@pytest.mark.parametrize("new,wide", [([3, 2, 1], 0), ([100, 130, 1], 1024)])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (1, 0), (100, 0), (127, 40), (2 ** 30, 3)])
def test_attention(make, run, new, wide, window, n_sink):
    total = [320, 336, 333]
    bt = make(new, total, Hq=8, Hkv=1, D=128, seed=3, extra_width=wide)
    far = 16 * bt.table.shape[1] + new[1] + (window if window < 2 ** 30 else 0)   # the first row is past the table and the window
    bt.kv_len[1] = far
    want, want_lse, st = run(bt, window, n_sink, max_q_len=max(new))
    assert st == BOUNDS
    assert (want_lse[3 if new[1] == 2 else 100] == -np.inf).all() == (window in (1, 100))   # they see sinks, or all there is
    for end in (TOP, TOP - 1, TOP - 100, TOP - 128) if window < 2 ** 30 else (2 ** 30 + 1,):
        bt.kv_len[1] = end
        out, lse, st = run(bt, window, n_sink, max_q_len=max(new))
        assert st == BOUNDS
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)
