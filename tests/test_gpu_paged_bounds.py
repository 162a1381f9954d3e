"""Page ids outside the cache in moe_paged_attention (include/paged_kv.h): they
are reported, and their positions are as if the rows did not see them.

The request concerned is compared with fp64 attention over its other
positions, within the bounds of the other attention tests: the f16 weights and
fp32 scores move a row by at most 2^-10 max|v|, bf16 rounds it once."""
import math

import numpy as np
import pytest

from oracle import decode_oracle as do
from tests.decode_util import Batch, values64
from tests.test_gpu_paged_kv import run_attention

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def without(bt, b, hidden):
    """fp64 (out, lse) of request b, whose positions `hidden` nobody sees."""
    c, n, total, group = bt.oracle_cache(), int(bt.cu[b + 1] - bt.cu[b]), int(bt.kv_len[b]), bt.Hq // bt.Hkv
    q = values64(bt.q)[bt.cu[b]:bt.cu[b + 1]]
    out, lse = np.zeros_like(q), np.full(q.shape[:2], -math.inf)
    shown = np.array([j not in hidden for j in range(total)])
    for h in range(bt.Hkv):
        K, V = c.values("k", b, h, total), c.values("v", b, h, total)
        for i in range(n):
            see = shown & (np.arange(total) <= total - n + i)
            if not see.any():
                continue
            for hq in range(h * group, (h + 1) * group):
                z = bt.D ** -0.5 * (K[see] @ q[i, hq])
                e = np.exp(z - z.max())
                out[i, hq], lse[i, hq] = (e / e.sum()) @ V[see], z.max() + math.log(e.sum())
    vmax = np.max(np.abs(np.nan_to_num(do.decode_e4m3(bt.codes["v"]))) * bt.scales["v"][:, :, None, None])
    return out, lse, vmax


def compare(got_o, got_l, ref_o, ref_l, vmax):
    live = ref_l > -math.inf
    assert np.all(got_o[..., ~live, :] == 0.0) and np.all(got_l[..., ~live] == -math.inf)
    assert np.all(np.abs(got_o - ref_o) <= 2.0 ** -8 * np.abs(ref_o) + 2.0 ** -10 * vmax)
    assert np.all(np.abs(got_l[..., live] - ref_l[live]) <= 2e-5 * (1 + np.max(np.abs(ref_l[live]), initial=0.0)))


def spoil(bt, pages, bad):
    """Gives page-table entries of request 0 the id `bad`; the positions concerned."""
    hidden = set()
    for p in pages:
        bt.table[0, p] = bt.n_pages if bad is None else bad
        hidden |= set(range(p * bt.page, (p + 1) * bt.page))
    return hidden


@pytest.mark.parametrize("bad", [-1, None, LOW, HIGH])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_few_rows(D, bad):
    bt = Batch([1, 2], [100, 60], Hq=8, Hkv=2, D=D, seed=31)
    ref = without(bt, 0, spoil(Batch([1], [100]), [2, 6], -1))
    other = without(bt, 1, set())
    spoil(bt, [2, 6], bad)
    out, lse, st = run_attention(bt)
    assert st == 6                                        # MOE_ERR_DEVICE_BOUNDS
    compare(values64(out)[:1], values64(lse)[:1], *ref)
    compare(values64(out)[1:], values64(lse)[1:], *other)


@pytest.mark.parametrize("bad", [-1, LOW])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_few_rows_after_other_pages(D, bad):
    """Long pieces of many requests: what was fetched for earlier pages is still there when a bad id is met."""
    bt = Batch([2], [1500], Hq=4, Hkv=1, D=D, seed=32)
    pages = [0, 20, 41, 42, 43, 44, 93]
    ref = without(bt, 0, spoil(Batch([2], [1500]), pages, -1))
    spoil(bt, pages, bad)
    bt.B, bt.T = 900, 1800
    bt.q = bt.q.repeat(900, 1, 1)
    bt.cu = np.arange(0, 1801, 2).astype(np.int32)
    bt.kv_len = np.full(900, 1500, dtype=np.int32)
    bt.table = np.repeat(bt.table, 900, 0)
    out, lse, st = run_attention(bt, max_q_len=2)
    assert st == 6
    compare(values64(out).reshape(900, 2, 4, D), values64(lse).reshape(900, 2, 4), *ref)


@pytest.mark.parametrize("bad", [-1, None, LOW, HIGH])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows(D, bad):
    bt = Batch([100, 160], [1000, 900], Hq=8, Hkv=2, D=D, seed=33, extra_width=1024)
    pages = [0, 2, 8, 9, 10, 11, 12, 13, 14, 15, 62]      # a whole step among them
    ref = without(bt, 0, spoil(Batch([100], [1000]), pages, -1))
    other = without(bt, 1, set())
    spoil(bt, pages, bad)
    for hint in (0, 160):
        out, lse, st = run_attention(bt, max_q_len=hint)
        assert st == 6
        compare(values64(out)[:100], values64(lse)[:100], *ref)
        compare(values64(out)[100:], values64(lse)[100:], *other)


@pytest.mark.parametrize("new,wide", [(3, 0), (150, 1024)])
def test_rows_whose_every_page_is_gone(new, wide):
    """A prompt whose first pages are bad: its first rows see nothing."""
    bt = Batch([new], [new], Hq=8, Hkv=1, seed=34, extra_width=wide)
    pages = [0] if new == 3 else [0, 1]
    ref = without(bt, 0, spoil(Batch([new], [new]), pages, -1))
    assert not np.all(ref[1] > -math.inf)
    for bad in (-1, LOW):
        spoil(bt, pages, bad)
        out, lse, st = run_attention(bt, max_q_len=new)
        assert st == 6
        compare(values64(out), values64(lse), *ref)
