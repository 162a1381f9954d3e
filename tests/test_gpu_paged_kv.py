"""GPU parity of moe_kv_append and moe_paged_attention (include/paged_kv.h)
against the fp64 oracle.

Append.  A stored code is the nearest E4M3 value to y / s: it may be off by
half a step, 2^-4 of the value's size (2^-10 below the normal range), plus the
fp32 error of norm and rotation, about 1e-6 of the row's largest element, for
which 1e-5 is allowed.  Page scales are exact powers of two and have to be
equal.  q_out: one bf16 rounding (2^-9) and the same fp32 error.

Attention.  The weights are rounded to f16 (2^-11 relative, those below the
f16 range to nothing), so a sum of them moves by at most 2^-11 max|v|; the
fp32 scores move it by about 1e-5 max|v| more; the output is rounded to bf16
once (2^-9).  Twice that is allowed: 2^-8 |ref| + 2^-10 max|v|.  lse: the
fp32 sum of 64..256 products, each of which may be off by 2^-24 of the sum of
sizes, so 2e-5 (1 + max|z|)."""
import math

import numpy as np
import pytest
import torch

from oracle import decode_oracle as do
from tests.decode_util import Batch, codes_of, values64
from top_routed_expert_gb300 import abi

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- append

def run_append(bt, rot, layout, norm, with_q=True, positions=None, n_pos=None, joint=False, stream=None, cs=None):
    dev = "cuda"
    rng = np.random.default_rng(7)
    n_pos = max(bt.total) + 3 if n_pos is None else n_pos
    gq = rng.uniform(0.5, 1.5, bt.D).astype(np.float32) if norm else None
    gk = rng.uniform(0.5, 1.5, bt.D).astype(np.float32) if norm else None
    if rot and cs is None:
        i = np.arange(rot // 2)
        ang = np.arange(n_pos)[:, None] * 10000.0 ** (-2.0 * i / rot)
        cs = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    kc, vc, ks, vs, table, cache = bt.device()
    if joint:   # slices of one projection's output, with a gap behind them
        x = torch.cat([bt.q.flatten(1), bt.k.flatten(1), bt.v.flatten(1), torch.zeros(bt.T, 8, dtype=torch.bfloat16)], 1).to(dev)
        a, b, c = bt.Hq * bt.D, (bt.Hq + bt.Hkv) * bt.D, (bt.Hq + 2 * bt.Hkv) * bt.D
        q, k, v = (y.unflatten(1, (-1, bt.D)) for y in (x[:, :a], x[:, a:b], x[:, b:c]))
    else:
        q, k, v = bt.q.to(dev), bt.k.to(dev), bt.v.to(dev)
    q_out = torch.full((bt.T, bt.Hq, bt.D), 5.0, dtype=torch.bfloat16, device=dev)
    if not with_q:
        q = q_out = None
    cu, kv_len = bt.lengths()
    cfg = abi.make_kv_append_config(q, k, v, q_out, bt.B, rot_dim=rot, n_pos=n_pos,
                                    rope_layout=abi.MOE_ROPE_HALF if layout == "half" else abi.MOE_ROPE_INTERLEAVED)
    args = (cfg, cache, q, k, v, up(gq), up(gk), up(cs), up(positions), cu, kv_len, q_out)
    torch.cuda.synchronize()
    abi.moe_kv_append(*args, stream=stream)
    st = abi.moe_get_device_status(stream)
    torch.cuda.synchronize()
    ref = bt.oracle_cache()
    return dict(q_out=q_out, kc=kc, vc=vc, ks=ks, vs=vs, st=st, ref=ref, gq=gq, gk=gk, cs=cs, args=args)


def check_append(bt, r, layout, positions=None):
    ref = r["ref"]
    before = {n: bt.codes[n].copy() for n in ("k", "v")}
    q_ref, exact = do.kv_append(ref, None if r["q_out"] is None else values64(bt.q), values64(bt.k), values64(bt.v),
                                r["gq"], r["gk"], r["cs"], positions, bt.cu, bt.kv_len, layout)
    assert r["st"] == 0
    if q_ref is not None:
        got = values64(r["q_out"])
        bound = 2.0 ** -8 * np.abs(q_ref) + 1e-5 * np.max(np.abs(q_ref), axis=-1, keepdims=True)
        assert np.all(np.abs(got - q_ref) <= bound)
    for name, codes, scale in (("k", r["kc"], r["ks"]), ("v", r["vc"], r["vs"])):
        assert np.array_equal(scale.cpu().numpy().astype(np.float64), ref.scale[name])
        got = values64(codes)
        fresh = np.zeros(got.shape[:3], dtype=bool)
        for page, head, slot, x in exact[name]:
            fresh[page, head, slot] = True
            bound = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) + 1e-5 * np.max(np.abs(x))
            assert np.all(np.abs(got[page, head, slot] - x) <= bound), (name, page, head, slot)
        # tokens that were there: re-rounded codes or the same ones, as the oracle has them
        same = np.array_equal(got[~fresh], ref.codes[name][~fresh], equal_nan=True)
        assert same
        untouched = np.all((ref.codes[name] == do.decode_e4m3(before[name])) | np.isnan(ref.codes[name]), axis=3) & ~fresh
        assert np.array_equal(codes_of(codes)[untouched], before[name][untouched])


@pytest.mark.parametrize("new,total,kw,rot,layout,norm", [
    ([1], [1], dict(), 128, "half", True),
    ([1, 1, 1, 1, 1], [1, 16, 17, 32, 100], dict(), 128, "half", True),
    ([5, 0, 33, 1], [5, 40, 50, 64], dict(order="nhd"), 128, "half", False),
    ([37, 16], [53, 32], dict(D=64, page=32, Hq=6, Hkv=3), 32, "interleaved", True),
    ([130, 3], [131, 129], dict(D=64, page=128, Hq=4, Hkv=4), 64, "half", True),
    ([70, 2], [100, 2], dict(D=256, page=64, Hq=2, Hkv=1), 192, "interleaved", False),
    ([140], [150], dict(D=256, page=128, Hq=3, Hkv=1), 256, "half", True),
    ([20, 9], [21, 30], dict(D=128, page=64, order="nhd"), 0, "half", False),
    ([7, 7, 7], [23, 7, 12], dict(D=128, page=16), 8, "interleaved", True),
])
@pytest.mark.parametrize("joint", [False, True])
def test_append(new, total, kw, rot, layout, norm, joint):
    bt = Batch(new, total, seed=len(new) + rot, **kw)
    check_append(bt, run_append(bt, rot, layout, norm, joint=joint), layout)


def test_append_without_queries_and_with_positions():
    bt = Batch([9, 4], [30, 4], seed=3)
    pos = np.array([3, 1, 4, 1, 5, 9, 2, 6, 5, 0, 33, 8, 7], dtype=np.int32)
    r = run_append(bt, 64, "half", True, with_q=False, positions=pos, n_pos=34)
    check_append(bt, r, "half", positions=pos)


def test_append_queries_in_place():
    bt = Batch([5, 1], [21, 9], seed=4)
    ref = run_append(bt, 128, "half", True)
    r = run_append(bt, 128, "half", True)
    q = bt.q.cuda()
    cfg, cache = r["args"][:2]
    abi.moe_kv_append(cfg, cache, q, *r["args"][3:11], q)
    assert torch.equal(q, ref["q_out"])


def test_append_again_changes_nothing_and_pieces_agree():
    """A call repeated leaves what it left; a prompt in pieces gives the scales
    of the whole and, with values well inside E4M3's normal range, its codes."""
    whole = Batch([41], [41], seed=5)
    for x in (whole.k, whole.v):   # sizes in [1/4, 4]: no code becomes subnormal when a scale grows
        x.copy_(torch.sign(x.float()) * (0.25 + 3.75 * torch.rand(x.shape, generator=torch.Generator().manual_seed(1))))
    a = run_append(whole, 0, "half", False)
    abi.moe_kv_append(*a["args"])
    once = codes_of(a["kc"]), codes_of(a["vc"])
    check_append(whole, a, "half")
    abi.moe_kv_append(*a["args"])
    assert np.array_equal(once[0], codes_of(a["kc"])) and np.array_equal(once[1], codes_of(a["vc"]))
    kc, vc, ks, vs, table, cache = whole.device()
    done = 0
    for n in (1, 15, 3, 20, 2):
        part = slice(done, done + n)
        k, v = whole.k[part].cuda(), whole.v[part].cuda()
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ln = torch.tensor([done + n], dtype=torch.int32, device="cuda")
        abi.moe_kv_append(abi.make_kv_append_config(None, k, v, None, 1), cache, None, k, v, None, None, None, None, cu,
                          ln, None)
        done += n
    assert np.array_equal(ks.cpu().numpy()[table.cpu().numpy()[0]], a["ks"].cpu().numpy()[whole.table[0]])
    live = [(whole.table[0, j // 16], slice(None), j % 16) for j in range(41)]
    for c, ref in ((kc, once[0]), (vc, once[1])):
        c = codes_of(c)
        assert all(np.array_equal(c[at], ref[at]) for at in live)


def test_append_zero_rows_and_tiny_values():
    bt = Batch([18], [18], seed=6)
    bt.k.zero_()
    bt.v.copy_(bt.v * 2.0 ** -60)
    check_append(bt, run_append(bt, 0, "half", False), "half")
    bt = Batch([18], [18], seed=6)
    bt.k.copy_(bt.k * 2.0 ** 110)    # scales far from 1 on both sides
    bt.v.copy_(bt.v * 2.0 ** -30)
    check_append(bt, run_append(bt, 0, "half", False), "half")


def test_append_nonfinite_elements():
    bt = Batch([20, 6], [20, 22], seed=8)
    bt.k[3, 1, 17] = math.nan
    bt.v[21, 0, 5] = math.inf
    bt.v[22, 0, 6] = -math.inf
    r = run_append(bt, 0, "half", False)
    assert r["st"] == 8                                   # MOE_ERR_DEVICE_NONFINITE
    do.kv_append(r["ref"], None, values64(bt.k), values64(bt.v), None, None, None, None, bt.cu, bt.kv_len)
    for name, codes, scale in (("k", r["kc"], r["ks"]), ("v", r["vc"], r["vs"])):
        assert np.array_equal(scale.cpu().numpy(), r["ref"].scale[name])
        assert np.array_equal(values64(codes), r["ref"].codes[name], equal_nan=True)   # no rotation: bit for bit


@pytest.mark.parametrize("fault", ["page_low", "page_high", "table_short", "position", "cu_drop", "cu_high", "len"])
def test_append_bounds_are_reported_and_contained(fault):
    bt = Batch([6, 20, 5], [6, 40, 21], seed=9)
    good = run_append(bt, 128, "half", True)
    used = set(bt.table[bt.table >= 0].ravel().tolist())
    n_pos, positions = None, None
    if fault == "page_low":
        bt.table[1, 1] = -1
    elif fault == "page_high":
        bt.table[1, 1] = bt.n_pages
    elif fault == "table_short":
        bt.kv_len[1] += 16 * bt.table.shape[1]
        n_pos = 4096
    elif fault == "position":
        positions = np.zeros(bt.T, dtype=np.int32)
        positions[[7, 9]] = [-1, 4096]
        n_pos = 4096
    elif fault == "cu_drop":
        bt.cu[2] = 4
    elif fault == "cu_high":
        bt.cu[3] = bt.T + 7
    elif fault == "len":
        bt.kv_len[1] = 3
    r = run_append(bt, 128, "half", True, n_pos=n_pos, positions=positions)
    assert r["st"] == 6                                   # MOE_ERR_DEVICE_BOUNDS
    assert abi.moe_get_device_status() == 0
    if fault in ("page_low", "page_high", "cu_high", "len"):
        # the first request is whole, and nothing lies outside the requests' pages
        for c, ref in ((r["kc"], good["kc"]), (r["vc"], good["vc"])):
            a, b = codes_of(c), codes_of(ref)
            assert np.array_equal(a[bt.table[0, 0]], b[bt.table[0, 0]])
            assert np.all(a[[p for p in range(bt.n_pages) if p not in used]] == 0x7F)
    if fault == "position":
        assert np.all(values64(r["q_out"])[[7, 9]] == 5.0)
        assert np.all(values64(r["q_out"])[8] != 5.0)


# ----------------------------------------------------------------- attention

def run_attention(bt, window=0, n_sink=0, sm_scale=None, max_q_len=0, lse=True, stream=None, q=None):
    kc, vc, ks, vs, table, cache = bt.device()
    q = bt.q.cuda() if q is None else q
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda") if lse else None
    cu, kv_len = bt.lengths()
    cfg = abi.make_paged_attention_config(q, out, bt.B, max_q_len=max_q_len, window=window, n_sink=n_sink,
                                          sm_scale=sm_scale)
    ws = torch.full((abi.moe_paged_attention_ws_bytes(cfg, cache),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    abi.moe_paged_attention(cfg, cache, q, cu, kv_len, out, ls, ws, stream=stream)
    st = abi.moe_get_device_status(stream)
    return out, ls, st


def check_attention(bt, window=0, n_sink=0, rows=None, **kw):
    out, lse, st = run_attention(bt, window, n_sink, **kw)
    assert st == 0
    ref_o, ref_l = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5, window, n_sink)
    rows = slice(None) if rows is None else rows
    got_o, got_l = values64(out)[rows], values64(lse)[rows]
    ref_o, ref_l = ref_o[rows], ref_l[rows]
    live = ref_l > -math.inf
    assert np.all(got_l[~live] == -math.inf) and np.all(got_o[~live] == 0.0)
    vmax = max(np.nanmax(np.abs(do.decode_e4m3(bt.codes["v"])) * bt.scales["v"][:, :, None, None], initial=0.0), 1e-30)
    assert np.all(np.abs(got_o - ref_o) <= 2.0 ** -8 * np.abs(ref_o) + 2.0 ** -10 * vmax)
    assert np.all(np.abs(got_l[live] - ref_l[live]) <= 2e-5 * (1 + np.max(np.abs(ref_l[live]), initial=0.0)))
    return out, lse


SHAPES = [
    ([1], [1], dict()),
    ([1], [129], dict(Hq=32, Hkv=4)),
    ([1, 1, 1, 1], [15, 16, 17, 300], dict(Hq=7, Hkv=1)),
    ([1, 1], [65, 63], dict(Hq=2, Hkv=2, order="nhd")),
    ([1, 3, 0, 2], [40, 3, 50, 90], dict(Hq=16, Hkv=1, page=32)),
    ([2, 17], [200, 30], dict(Hq=3, Hkv=3, D=64, page=64)),
    ([1, 5], [130, 128], dict(Hq=40, Hkv=2, D=64, page=128, order="nhd")),
    ([3, 1], [70, 31], dict(Hq=4, Hkv=2, D=256, page=16)),
    ([33], [33], dict(Hq=2, Hkv=1, D=256, page=64)),
    ([150, 40], [150, 230], dict(Hq=8, Hkv=1, page=16)),
    ([70, 1, 129], [90, 77, 129], dict(Hq=4, Hkv=4, page=32, order="nhd")),
    ([40], [300], dict(Hq=14, Hkv=2, D=64, page=16)),
]


@pytest.mark.parametrize("new,total,kw", SHAPES)
@pytest.mark.parametrize("hint", [False, True])
def test_attention(new, total, kw, hint):
    bt = Batch(new, total, seed=sum(total), **kw)
    check_attention(bt, max_q_len=max(new) if hint else 0)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (16, 4), (40, 0), (64, 70), (129, 5), (10 ** 6, 3)])
@pytest.mark.parametrize("new,total,kw", [SHAPES[2], SHAPES[5], SHAPES[9], SHAPES[7]])
def test_attention_window(new, total, kw, window, n_sink):
    bt = Batch(new, total, seed=window + n_sink, **kw)
    check_attention(bt, window, n_sink, max_q_len=max(new))


def test_attention_evicted_pages():
    """Pages that a window has left behind may be gone from the table, and hold anything."""
    bt = Batch([1, 4, 60], [200, 300, 260], Hq=8, Hkv=1, seed=11)
    window, n_sink = 50, 4
    ref = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5, window, n_sink)
    for b in range(bt.B):
        first = bt.total[b] - bt.new[b]
        for pg in range(1, (first - window + 1) // bt.page):
            bt.codes["k"][bt.table[b, pg]] = 0x7F
            bt.codes["v"][bt.table[b, pg]] = 0xFF
            bt.scales["k"][bt.table[b, pg]] = math.nan
            bt.table[b, pg] = -1
    for hint in (0, 60):
        out, lse, st = run_attention(bt, window, n_sink, max_q_len=hint)
        assert st == 0
        assert np.max(np.abs(values64(out) - ref[0])) <= 2.0 ** -8 * np.max(np.abs(ref[0])) + 2.0 ** -10 * 32
        assert np.max(np.abs(values64(lse) - ref[1])) <= 2e-5 * (1 + np.max(np.abs(ref[1])))


def test_attention_rows_that_see_nothing():
    # kv_len below the new tokens, zero and negative
    bt = Batch([5, 3, 2, 130], [5, 3, 2, 130], Hq=8, Hkv=1, seed=12)
    bt.kv_len[:] = [2, 0, -7, 100]
    for hint in (0, 130):
        out, lse = check_attention(bt, max_q_len=hint)
        assert np.all(values64(out)[:3] == 0.0) and np.all(values64(lse)[5:10] == -math.inf)


def test_attention_nan_query_stays_in_its_row():
    for new, total in (([2, 1], [70, 40]), ([140], [150])):
        bt = Batch(new, total, Hq=8, Hkv=2, seed=13)
        clean_o, clean_l, _ = run_attention(bt, max_q_len=max(new))
        bt.q[1, 3, 5], bt.q[0, 6, 0] = math.nan, math.inf
        out, lse, _ = run_attention(bt, max_q_len=max(new))
        bad = np.zeros((bt.T, 8), dtype=bool)
        bad[1, 3] = bad[0, 6] = True
        assert np.all(np.isnan(values64(out)[bad])) and np.all(np.isnan(values64(lse)[bad]))
        assert np.array_equal(values64(out)[~bad], values64(clean_o)[~bad])
        assert np.array_equal(values64(lse)[~bad], values64(clean_l)[~bad])


def test_attention_extreme_scales_and_scores():
    """Page scales from 2^-40 to 2^40, and scores of a few thousand."""
    for new, total in (([2, 1], [70, 100]), ([130], [140])):
        bt = Batch(new, total, Hq=8, Hkv=2, seed=14)
        n = bt.scales["v"].shape[0]
        bt.scales["v"] = 2.0 ** np.linspace(-40, 0, n * 2).round().reshape(n, 2)
        check_attention(bt, max_q_len=max(new))
        bt.q.mul_(200.0)
        out, lse, st = run_attention(bt, max_q_len=max(new))
        ref_o, ref_l = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5)
        assert np.max(np.abs(values64(lse) - ref_l)) <= 2e-5 * (1 + np.max(np.abs(ref_l)))


def test_attention_pages_out_of_the_cache():
    bt = Batch([1, 2], [100, 60], seed=15)
    keep = bt.table.copy()
    bt.table[0, 2] = bt.n_pages
    out, lse, st = run_attention(bt)
    assert st == 6
    # the rest of the call is computed as without that page
    full = Batch([1, 2], [100, 60], seed=15)
    ref_o, _ = do.paged_attention(full.oracle_cache(), values64(full.q), full.cu, full.kv_len, full.D ** -0.5)
    assert np.max(np.abs(values64(out)[1:] - ref_o[1:])) <= 2.0 ** -8 * np.max(np.abs(ref_o)) + 2.0 ** -10 * 32
    bt.table[:] = keep
    bt.cu[1] = 9                                          # past T
    out, _, st = run_attention(bt)
    assert st == 6 and np.all(values64(out) == 7.0)


def test_attention_strided_rows_other_stream_and_no_lse():
    bt = Batch([2, 40], [33, 77], Hq=8, Hkv=2, seed=16)
    ref, ref_l, _ = run_attention(bt, max_q_len=40)
    wide = torch.zeros(bt.T, bt.Hq + 3, bt.D, dtype=torch.bfloat16, device="cuda")
    wide[:, :bt.Hq] = bt.q.cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, lse, st = run_attention(bt, max_q_len=40, stream=s, q=wide[:, :bt.Hq])
    s.synchronize()
    assert st == 0 and torch.equal(out, ref) and torch.equal(lse, ref_l)
    out, _, _ = run_attention(bt, max_q_len=40, lse=False)
    assert torch.equal(out, ref)


def test_attention_same_bits_every_time():
    bt = Batch([1, 1, 3, 90], [700, 33, 260, 400], Hq=8, Hkv=2, seed=17)
    a = run_attention(bt, max_q_len=90)
    for _ in range(3):
        b = run_attention(bt, max_q_len=90)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# Enough rows, and a page table wide enough, for the tensor-memory kernel, and
# contexts long enough that it cuts
# row blocks along the cached tokens; the third and the last mix both kernels, the
# fourth and fifth have equal prompts.
WIDE = dict(extra_width=1024)
MANY = [
    ([64, 130], [900, 130], dict(Hq=16, Hkv=2)),
    ([300], [1500], dict(Hq=7, Hkv=1, D=64, page=64)),
    ([1, 100, 0, 3], [700, 2100, 40, 5], dict(Hq=32, Hkv=4, page=32, order="nhd")),
    ([128, 128], [128, 1000], dict(Hq=8, Hkv=8)),
    ([65] * 4, [65, 770, 769, 66], dict(Hq=8, Hkv=8, D=64, page=128)),
    ([1] * 6 + [100] + [1] * 6, [1700] * 6 + [400] + [1700] * 6, dict(Hq=32, Hkv=8, D=64, page=64)),
]


@pytest.mark.parametrize("new,total,kw", MANY)
@pytest.mark.parametrize("hint", [False, True])
def test_attention_many_rows(new, total, kw, hint):
    bt = Batch(new, total, seed=sum(total), **WIDE, **kw)
    check_attention(bt, max_q_len=max(new) if hint else 0)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (130, 4), (800, 0), (900, 300), (10 ** 6, 3)])
@pytest.mark.parametrize("new,total,kw", MANY[:3])
def test_attention_many_rows_window(new, total, kw, window, n_sink):
    bt = Batch(new, total, seed=window + n_sink, **WIDE, **kw)
    check_attention(bt, window, n_sink, max_q_len=max(new))


def test_attention_many_rows_evicted_pages():
    bt = Batch([100, 64, 150], [1900, 300, 1260], Hq=8, Hkv=1, seed=21, **WIDE)
    window, n_sink = 900, 4
    ref = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5, window, n_sink)
    for b in range(bt.B):
        first = bt.total[b] - bt.new[b]
        for pg in range(1, (first - window + 1) // bt.page):
            bt.codes["k"][bt.table[b, pg]] = 0x7F
            bt.codes["v"][bt.table[b, pg]] = 0xFF
            bt.scales["k"][bt.table[b, pg]] = math.nan
            bt.table[b, pg] = -1
    out, lse, st = run_attention(bt, window, n_sink, max_q_len=150)
    assert st == 0
    assert np.max(np.abs(values64(out) - ref[0])) <= 2.0 ** -8 * np.max(np.abs(ref[0])) + 2.0 ** -10 * 32
    assert np.max(np.abs(values64(lse) - ref[1])) <= 2e-5 * (1 + np.max(np.abs(ref[1])))


def test_attention_many_rows_that_see_nothing():
    bt = Batch([50, 100, 60, 300], [50, 100, 60, 1300], Hq=8, Hkv=1, seed=22, **WIDE)
    bt.kv_len[:] = [20, 0, -7, 1100]
    for hint in (0, 300):
        out, lse = check_attention(bt, max_q_len=hint)
        assert np.all(values64(out)[:30] == 0.0) and np.all(values64(lse)[50:210] == -math.inf)


def test_attention_many_rows_nan_query_stays_in_its_row():
    bt = Batch([260], [1150], Hq=8, Hkv=2, seed=23, **WIDE)
    clean_o, clean_l, _ = run_attention(bt)
    bt.q[1, 3, 5], bt.q[0, 6, 0], bt.q[259, 0, 127] = math.nan, math.inf, -math.inf
    out, lse, _ = run_attention(bt)
    bad = np.zeros((bt.T, 8), dtype=bool)
    bad[1, 3] = bad[0, 6] = bad[259, 0] = True
    assert np.all(np.isnan(values64(out)[bad])) and np.all(np.isnan(values64(lse)[bad]))
    assert np.array_equal(values64(out)[~bad], values64(clean_o)[~bad])
    assert np.array_equal(values64(lse)[~bad], values64(clean_l)[~bad])


def test_attention_many_rows_extreme_scales_and_scores():
    bt = Batch([256], [1140], Hq=8, Hkv=2, seed=24, **WIDE)
    n = bt.scales["v"].shape[0]
    bt.scales["v"] = 2.0 ** np.linspace(-40, 0, n * 2).round().reshape(n, 2)
    check_attention(bt)
    bt.q.mul_(200.0)
    out, lse, st = run_attention(bt)
    ref_o, ref_l = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5)
    assert np.max(np.abs(values64(lse) - ref_l)) <= 2e-5 * (1 + np.max(np.abs(ref_l)))


def test_attention_many_rows_page_out_of_the_cache():
    bt = Batch([100, 160], [1000, 900], Hq=8, Hkv=2, seed=25, **WIDE)
    full = Batch([100, 160], [1000, 900], Hq=8, Hkv=2, seed=25, **WIDE)
    bt.table[0, 2] = bt.n_pages
    out, lse, st = run_attention(bt)
    assert st == 6
    ref_o, _ = do.paged_attention(full.oracle_cache(), values64(full.q), full.cu, full.kv_len, full.D ** -0.5)
    assert np.max(np.abs(values64(out)[100:] - ref_o[100:])) <= 2.0 ** -8 * np.max(np.abs(ref_o)) + 2.0 ** -10 * 32


def test_attention_offsets_that_name_rows_again():
    """Offsets out of order are reported; requests that overlap make no more work than the rows have."""
    bt = Batch([300], [1100], Hq=8, Hkv=1, seed=27, **WIDE)
    ref, _, _ = run_attention(bt)
    bt.B = 101
    bt.cu = np.array([0, 300] * 51, dtype=np.int32)
    bt.kv_len = np.full(101, 1100, dtype=np.int32)
    bt.table = np.repeat(bt.table, 101, 0)
    out, _, st = run_attention(bt)
    assert st == 6
    # every request that names a row has the same result for it, within twice the bound above (|v| <= 448 / 32)
    got, ref = values64(out), values64(ref)
    assert np.all(np.abs(got - ref) <= 2.0 ** -7 * np.abs(ref) + 2.0 ** -9 * 14)


def test_attention_many_rows_same_bits_strided_other_stream():
    bt = Batch([1, 256, 3, 90], [1700, 1333, 260, 900], Hq=8, Hkv=2, seed=26, **WIDE)
    ref, ref_l, st = run_attention(bt, max_q_len=256)
    assert st == 0
    for _ in range(3):
        out, lse, _ = run_attention(bt, max_q_len=256)
        assert torch.equal(out, ref) and torch.equal(lse, ref_l)
    out, _, _ = run_attention(bt, max_q_len=256, lse=False)
    assert torch.equal(out, ref)
    wide = torch.zeros(bt.T, bt.Hq + 3, bt.D, dtype=torch.bfloat16, device="cuda")
    wide[:, :bt.Hq] = bt.q.cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, lse, st = run_attention(bt, max_q_len=256, stream=s, q=wide[:, :bt.Hq])
    s.synchronize()
    assert st == 0 and torch.equal(out, ref) and torch.equal(lse, ref_l)


def test_append_then_attend_in_a_graph():
    """Both calls captured on a side stream and replayed on new inputs."""
    bt = Batch([1, 1, 1], [20, 1, 50], Hq=8, Hkv=2, seed=18)
    kc, vc, ks, vs, table, cache = bt.device()
    q, k, v = bt.q.cuda(), bt.k.cuda(), bt.v.cuda()
    qo, out = torch.empty_like(q), torch.empty_like(q)
    cu, kv_len = bt.lengths()
    i = np.arange(64)
    ang = np.arange(64)[:, None] * 10000.0 ** (-i / 64)
    cs = torch.from_numpy(np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)).cuda()
    ca = abi.make_kv_append_config(q, k, v, qo, bt.B, rot_dim=128, n_pos=64)
    cp = abi.make_paged_attention_config(qo, out, bt.B, max_q_len=1)
    ws = torch.empty(abi.moe_paged_attention_ws_bytes(cp, cache), dtype=torch.uint8, device="cuda")

    def step():
        abi.moe_kv_append(ca, cache, q, k, v, None, None, cs, None, cu, kv_len, qo)
        abi.moe_paged_attention(cp, cache, qo, cu, kv_len, out, None, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    kv_len += 1                                           # the next token of every request
    q.copy_(q.flip(0)), k.copy_(k * 0.5), v.copy_(v.flip(0))
    saved = [x.clone() for x in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    for x, y in zip((kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), saved):
        x.copy_(y)
    step()
    assert abi.moe_get_device_status() == 0 and torch.equal(got, out)


def test_attention_long_cache_past_32_bit_offsets():
    """A cache of over 4 GB: byte offsets need 64 bits."""
    D, page, n_pages = 128, 128, 280_000                  # 4.6 GB of keys, the same of values
    k = torch.zeros(n_pages, 1, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.zeros(n_pages, 1, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks = torch.full((n_pages, 1), 2.0 ** -6, device="cuda")
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32, device="cuda")
    cache = abi.make_kv_cache(k, v, ks, ks.clone(), table)
    g = torch.Generator().manual_seed(19)
    n = 300
    kn, vn = (torch.randn(n, 1, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(n, 4, D, generator=g).to(torch.bfloat16).cuda()
    qo, out = torch.empty_like(q), torch.empty_like(q)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    abi.moe_kv_append(abi.make_kv_append_config(q, kn, vn, qo, 1), cache, q, kn, vn, None, None, None, None, cu, ln, qo)
    cfg = abi.make_paged_attention_config(qo, out, 1, max_q_len=n)
    ws = torch.empty(abi.moe_paged_attention_ws_bytes(cfg, cache), dtype=torch.uint8, device="cuda")
    abi.moe_paged_attention(cfg, cache, qo, cu, ln, out, None, ws)
    assert abi.moe_get_device_status() == 0
    K = (k[table[0].long()].double() * cache.tensors[2][table[0].long()].double()[..., None, None]).reshape(-1, D)[:n]
    V = (v[table[0].long()].double() * cache.tensors[3][table[0].long()].double()[..., None, None]).reshape(-1, D)[:n]
    assert (K - kn[:, 0].double()).abs().max() <= 2.0 ** -4 * kn.double().abs().max()
    z = torch.einsum("thd,jd->htj", q.double(), K) * D ** -0.5
    z = z.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -math.inf)
    ref = torch.einsum("htj,jd->thd", torch.softmax(z, -1), V)
    assert torch.all((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * V.abs().max())
