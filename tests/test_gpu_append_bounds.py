"""What moe_kv_append (include/paged_kv.h) writes beside a fault: everything of
the tokens that are not concerned, bit for bit as without it, and nothing of
those that are."""
import numpy as np
import pytest
import torch

from tests.decode_util import Batch, codes_of
from tests.test_gpu_paged_kv import run_append
from top_routed_expert_gb300 import abi

pytestmark = pytest.mark.gpu

BOUNDS = 6   # MOE_ERR_DEVICE_BOUNDS
NEW, TOTAL = [6, 20, 5], [6, 40, 21]


def state(r):
    """Codes and scales as bytes."""
    return {"k": codes_of(r["kc"]), "v": codes_of(r["vc"]), "ks": r["ks"].cpu().numpy(), "vs": r["vs"].cpu().numpy()}


def before(bt):
    return {"k": bt.codes["k"], "v": bt.codes["v"], "ks": bt.scales["k"].astype(np.float32),
            "vs": bt.scales["v"].astype(np.float32)}


def pages_of(bt, b):
    return [int(p) for p in bt.table[b, :-(-TOTAL[b] // bt.page)]]


def same(a, b, pages):
    assert all(np.array_equal(a[n][pages], b[n][pages]) for n in a)


def q_rows(r):
    return r["q_out"].view(torch.int16).cpu().numpy()


LOW = -2 ** 31


@pytest.mark.parametrize("fault", ["page -1", "page n", "page low", "table_short", "cu_high", "len", "cu_drop"])
@pytest.mark.parametrize("kw", [dict(), dict(D=64, Hq=4, Hkv=4, order="nhd"), dict(D=256, Hq=2, Hkv=1)])
def test_other_tokens_are_written_and_nothing_else(fault, kw):
    bt = Batch(NEW, TOTAL, seed=41, **kw)
    want, was = run_append(bt, 64, "half", True), before(bt)
    good, untouched = state(want), set(range(bt.n_pages))
    own = [pages_of(bt, b) for b in range(3)]
    kept = {0: own[0], 1: own[1], 2: own[2]}            # pages that come out as without the fault
    n_pos, rows = None, [True] * 3                        # rows: requests whose queries are turned
    if fault.startswith("page"):
        # the second page of request 1, with its new tokens 16..31: the keys and values of those alone
        bt.table[1, 1] = {"page -1": -1, "page n": bt.n_pages, "page low": LOW}[fault]
        kept[1] = [p for i, p in enumerate(own[1]) if i != 1]
    elif fault == "table_short":
        bt.kv_len[1] += 16 * bt.table.shape[1]
        n_pos, kept[1], rows[1] = 4096, [], None          # its queries turn by other angles
    elif fault == "cu_high":
        bt.cu[3] = bt.T + 7
        kept[2], rows[2] = [], False
    elif fault == "len":
        bt.kv_len[1] = 3
        kept[1], rows[1] = [], False
    elif fault == "cu_drop":
        bt.cu[2] = 4                                      # request 1 ends before it begins, 2 has more rows than tokens
        kept, rows = {1: [], 2: []}, [None, False, False]   # of request 0 some may stay unwritten
    r = run_append(bt, 64, "half", True, n_pos=n_pos)
    assert r["st"] == BOUNDS and abi.moe_get_device_status() == 0
    got = state(r)
    for b, pages in kept.items():
        same(got, good, pages)
        untouched -= set(pages)
    if fault == "cu_drop":
        untouched -= set(own[0])
        for p in own[0]:
            for n in got:
                assert np.all((got[n][p] == good[n][p]) | (got[n][p] == was[n][p]))
    same(got, was, sorted(untouched))
    for b, turned in enumerate(rows):
        at = slice(sum(NEW[:b]), sum(NEW[:b + 1]))
        if turned:
            assert np.array_equal(q_rows(r)[at], q_rows(want)[at])
        elif turned is False:
            assert torch.all(r["q_out"][at] == 5.0)       # as it was before the call


def test_tokens_with_an_angle_outside_the_table():
    """Two tokens of a page that also holds earlier ones: their slots stay, the scale is that of the others."""
    bt = Batch(NEW, TOTAL, seed=42)
    was = before(bt)
    pos = np.zeros(bt.T, dtype=np.int32)
    pos[[7, 9]] = [-1, 64]
    r = run_append(bt, 64, "half", True, positions=pos, n_pos=64)
    assert r["st"] == BOUNDS
    ref = Batch(NEW, TOTAL, seed=42)
    ref.k[[7, 9]], ref.v[[7, 9]] = 0, 0                   # as if they had no size
    want = run_append(ref, 64, "half", True, positions=np.zeros(bt.T, dtype=np.int32), n_pos=64)
    got, good = state(r), state(want)
    page = bt.table[1, 1]
    for n in ("k", "v"):
        for slot in (5, 7):                               # positions 21 and 23
            assert np.array_equal(got[n][page, :, slot], was[n][page, :, slot])
            good[n][page, :, slot] = was[n][page, :, slot]
    same(got, good, list(range(bt.n_pages)))
    keep = np.ones(bt.T, dtype=bool)
    keep[[7, 9]] = False
    assert np.array_equal(q_rows(r)[keep], q_rows(want)[keep]) and torch.all(r["q_out"][[7, 9]] == 5.0)
