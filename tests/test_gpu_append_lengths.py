"""Lengths near 2^31 in moe_kv_append (include/paged_kv.h): every position of such
a request is past the page table, so the call reports it and leaves the pages
that the request has as they were; the other requests' are written."""
import numpy as np
import pytest

from tests.decode_util import Batch
from tests.test_gpu_append_bounds import before, q_rows, same, state
from tests.test_gpu_paged_kv import run_append

pytestmark = pytest.mark.gpu

BOUNDS, TOP = 6, 2 ** 31 - 1


@pytest.mark.parametrize("end", [TOP, TOP - 1, TOP - 15, TOP - 16, TOP - 127, TOP - 128, TOP - 140])
@pytest.mark.parametrize("n,kw,layout", [(1, dict(), "half"), (17, dict(D=64, page=64), "interleaved"), (300, dict(page=128, D=256, Hkv=1), "half")])
def test_append(n, end, kw, layout):
    bt = Batch([20, n, 3], [33, n, 18], seed=n, **kw)
    good, was = run_append(bt, 0, layout, True), before(bt)
    bt.kv_len[1] = end
    r = run_append(bt, 0, layout, True)
    assert r["st"] == BOUNDS
    pages = [[int(p) for p in bt.table[b, :-(-bt.total[b] // bt.page)]] for b in range(3)]
    got, want = state(r), state(good)
    same(got, want, pages[0] + pages[2])
    same(got, was, sorted(set(range(bt.n_pages)) - set(pages[0] + pages[2])))
    assert np.array_equal(q_rows(r), q_rows(good))      # the queries need no page
