"""Lengths near 2^31 over the paged 4-bit cache (include/block_kv.h): every
position of such a request is past the page table, so the call reports it and
leaves the request's slots (a read: its rows) as they were, and does the others."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from tests.block_util import BlockBatch
from tests.decode_util import values64
from tests.test_gpu_block_kv import BOUNDS, check_cache, run_append, run_read

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1
ENDS = [TOP, TOP - 1, TOP - 15, TOP - 16, TOP - 40]


def batch(n, end, page):
    """Requests 0 and 2 are good, request 1 has n tokens and ends at `end`."""
    bt = BlockBatch([20, n, 3], [33, n, 18], Hq=2, Hkv=3, D=128, page=page, seed=n)
    bt.kv_len[1] = end
    return bt


@pytest.mark.parametrize("end", ENDS)
@pytest.mark.parametrize("n,page,layout", [(1, 16, "half"), (17, 64, "interleaved"), (300, 128, "half")])
def test_append(n, end, page, layout):
    bt = batch(n, end, page)
    r = run_append(bt, layout=layout, norm=True)
    assert r["st"] == BOUNDS
    ref, written = bt.oracle_cache(), []
    for b in (0, 2):
        for i in range(bt.new[b]):
            t, pos = bt.cu[b] + i, bt.total[b] - bt.new[b] + i
            at, slot = bt.table[b, pos // page], pos % page
            for h in range(bt.Hkv):
                for name, row in (("k", bo.key_rows(values64(bt.k)[t, h], r["gk"], None, layout)), ("v", values64(bt.v)[t, h])):
                    ref.codes[name][at, h, slot], ref.scale[name][at, h, slot] = bo.quantise(row, ref.g[name])
                    written.append((name, at, h, slot))
    check_cache(bt, r, ref, written)
    assert torch.all(r["q_out"] != 5.0)      # the queries need no page


@pytest.mark.parametrize("end", ENDS)
@pytest.mark.parametrize("n,page", [(1, 16), (17, 64), (300, 128)])
def test_read(n, end, page):
    bt = batch(n, end, page)
    good, c = (slice(0, 20), slice(20 + n, 23 + n)), bt.oracle_cache()
    for dtype in (torch.bfloat16, torch.float32):
        outs, st = run_read(bt, dtype)
        assert st == BOUNDS
        for name, out in zip("kv", outs):
            assert torch.all(out[20:20 + n] == 9.0)
            for b, rows in zip((0, 2), good):
                want = np.stack([c.values(name, b, h, bt.total[b])[bt.total[b] - bt.new[b]:] for h in range(bt.Hkv)], 1)
                assert np.array_equal(values64(out[rows]), want)
