"""GPU parity of the 4-bit cache's operators (include/block_kv.h) against the
oracle.

Append: the header fixes the fp32 operations, so codes and scales have to be
the oracle's, every byte of the cache (a zero's sign apart), and nothing else
may change.  q_out: one bf16 rounding (2^-8) and fp32 norm and rotation, for
which 1e-5 of the row's largest element is allowed.

Attention: the products' operands are exact.  Weights are rounded to f16 (2^-11
relative, under 2^-22 of the largest by 2^-33 of it), which moves a row by at
most 2^-11 max|v|; the fp32 scores move it by about 1e-5 max|v| more; the output
is rounded to bf16 once (2^-8): 2^-8 |ref| + 2^-10 max|v|.  lse: the fp32 sum of
64 to 256 products, each off by up to 2^-24 of the sum of sizes: 2e-5 (1 +
max|lse|).

Read: exact."""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from oracle import decode_oracle as do
from tests.block_util import BlockBatch, angles, host
from tests.decode_util import values64
from top_routed_expert_gb300 import abi

pytestmark = pytest.mark.gpu

BOUNDS, NONFINITE = 6, 8


# ----------------------------------------------------------------- append

def run_append(bt, rot=0, layout="half", norm=False, with_q=True, positions=None, n_pos=None, joint=False, stream=None):
    rng = np.random.default_rng(7)
    n_pos = max(bt.total) + 3 if n_pos is None else n_pos
    gq, gk = (rng.uniform(0.5, 1.5, bt.D).astype(np.float32) if norm else None for _ in range(2))
    cs = angles(n_pos, rot) if rot else None
    up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    tensors, cache = bt.device()
    if joint:   # slices of one projection's output, with a gap behind them
        x = torch.cat([bt.q.flatten(1), bt.k.flatten(1), bt.v.flatten(1), torch.zeros(bt.T, 8, dtype=torch.bfloat16)], 1).cuda()
        a, b, c = bt.Hq * bt.D, (bt.Hq + bt.Hkv) * bt.D, (bt.Hq + 2 * bt.Hkv) * bt.D
        q, k, v = (y.unflatten(1, (-1, bt.D)) for y in (x[:, :a], x[:, a:b], x[:, b:c]))
    else:
        q, k, v = bt.q.cuda(), bt.k.cuda(), bt.v.cuda()
    q_out = torch.full((bt.T, bt.Hq, bt.D), 5.0, dtype=torch.bfloat16, device="cuda")
    if not with_q:
        q = q_out = None
    cfg = abi.make_kv_append_config(q, k, v, q_out, bt.B, rot_dim=rot, n_pos=n_pos,
                                    rope_layout=abi.MOE_ROPE_HALF if layout == "half" else abi.MOE_ROPE_INTERLEAVED)
    args = (cfg, cache, q, k, v, up(gq), up(gk), up(cs), up(positions), *bt.lengths(), q_out)
    torch.cuda.synchronize()
    abi.moe_blockkv_append(*args, stream=stream)
    st = abi.moe_get_device_status(stream)
    torch.cuda.synchronize()
    return dict(q_out=q_out, cache=tensors, st=st, gq=gq, gk=gk, cs=cs, args=args)


def check_cache(bt, r, ref, written):
    """Every byte: the written slots are the oracle's, the others as they were."""
    for i, name in enumerate("kv"):
        codes, scales = host(r["cache"][i]), host(r["cache"][2 + i])
        fresh = np.zeros(codes.shape[:3], dtype=bool)
        for n, page, head, slot in written:
            fresh[page, head, slot] |= n == name
        got = bo.BlockCache(codes, codes, scales, scales, bt.table)
        nan = np.isnan(ref.scale[name])
        assert np.array_equal(got.scale["k"][fresh], ref.scale[name][fresh], equal_nan=True)
        numbers = fresh[..., None] & ~np.repeat(nan, 16, -1)      # a NaN block's codes may be any
        assert np.array_equal(got.codes["k"][numbers], ref.codes[name][numbers])
        assert np.array_equal(codes[~fresh], bt.codes[name][~fresh]) and np.array_equal(scales[~fresh], bt.scales[name][~fresh])


def check_append(bt, r, layout="half", positions=None):
    ref = bt.oracle_cache()
    q = None if r["q_out"] is None else values64(bt.q)
    q_ref, written = bo.append(ref, q, values64(bt.k), values64(bt.v), r["gq"], r["gk"], r["cs"], positions, bt.cu, bt.kv_len, layout)
    assert r["st"] == 0
    if q_ref is not None:
        bound = 2.0 ** -8 * np.abs(q_ref) + 1e-5 * np.max(np.abs(q_ref), axis=-1, keepdims=True)
        assert np.all(np.abs(values64(r["q_out"]) - q_ref) <= bound)
    check_cache(bt, r, ref, written)


@pytest.mark.parametrize("new,total,kw,rot,layout,norm", [
    ([1], [1], dict(), 128, "half", True),
    ([1, 1, 1, 1, 1], [1, 16, 17, 32, 100], dict(Hq=32, Hkv=4), 128, "half", True),
    ([5, 0, 33, 1], [5, 40, 50, 64], dict(order="nhd"), 128, "half", False),
    ([37, 16], [53, 32], dict(D=64, page=32, Hq=6, Hkv=3), 32, "interleaved", True),
    ([130, 3], [131, 129], dict(D=64, page=128, Hq=4, Hkv=4), 24, "half", True),
    ([70, 2], [100, 2], dict(D=256, page=64, Hq=2, Hkv=1), 192, "interleaved", False),
    ([40], [50], dict(D=256, page=128, Hq=3, Hkv=1), 256, "half", True),
    ([20, 9], [21, 30], dict(D=128, page=64, order="nhd"), 0, "half", False),
    ([20, 9], [21, 30], dict(D=128, page=64, gk=2.0 ** -9, gv=2.0 ** 7), 0, "interleaved", True),
    ([7, 7, 7], [23, 7, 12], dict(D=128, page=16), 8, "interleaved", True),
    ([17, 31], [18, 33], dict(D=128, page=16), 8, "half", True),
    ([17, 31], [18, 33], dict(D=128, page=32, Hkv=5, Hq=5), 48, "half", True),
    ([17, 31], [18, 33], dict(D=256, page=16, Hkv=1, Hq=1), 40, "half", False),
])
@pytest.mark.parametrize("joint", [False, True])
def test_append(new, total, kw, rot, layout, norm, joint):
    bt = BlockBatch(new, total, seed=len(new) + rot, **kw)
    check_append(bt, run_append(bt, rot, layout, norm, joint=joint), layout)


@pytest.mark.parametrize("new,total,kw,rot,layout,norm", [
    ([270, 1], [285, 40], dict(Hq=5, Hkv=5, D=64), 24, "half", True),
    ([270, 1], [285, 40], dict(Hq=1, Hkv=6, D=64, page=32, order="nhd"), 40, "interleaved", True),
    ([1, 300], [17, 300], dict(Hq=2, Hkv=3, D=128, page=64), 128, "half", False),
    ([1, 300], [17, 300], dict(Hq=2, Hkv=1, D=128), 128, "interleaved", False),
    ([260], [263], dict(Hq=1, Hkv=2, D=256, page=128), 192, "half", True),
    ([260], [263], dict(Hq=1, Hkv=2, D=256), 72, "interleaved", True),
    ([1] * 257, [1 + 5 * i % 61 for i in range(257)], dict(Hq=2, Hkv=2, D=64), 64, "half", True),
])
def test_append_many_tokens(new, total, kw, rot, layout, norm):
    """Over 256 tokens a thread works on four heads at a time."""
    bt = BlockBatch(new, total, seed=rot, **kw)
    check_append(bt, run_append(bt, rot, layout, norm, joint=rot % 3 == 0), layout)


def test_append_without_queries_and_with_positions():
    bt = BlockBatch([9, 4], [30, 4], seed=3)
    pos = np.array([3, 1, 4, 1, 5, 9, 2, 6, 5, 0, 33, 8, 7], dtype=np.int32)
    check_append(bt, run_append(bt, 64, "half", True, with_q=False, positions=pos, n_pos=34), positions=pos)


def test_append_queries_in_place_and_on_another_stream():
    bt = BlockBatch([5, 1], [21, 9], seed=4)
    ref = run_append(bt, 128, "half", True)
    s = torch.cuda.Stream()
    r = run_append(bt, 128, "half", True, stream=s)
    assert torch.equal(r["q_out"], ref["q_out"])
    check_append(bt, r)
    q = bt.q.cuda()
    abi.moe_blockkv_append(*r["args"][:2], q, *r["args"][3:11], q)
    assert torch.equal(q, ref["q_out"])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_a_prompt_in_pieces_is_the_prompt(layout):
    """Scales belong to a token: the same bytes however the prompt is cut."""
    bt = BlockBatch([41], [41], seed=5)
    whole = run_append(bt, 128, layout, True)
    check_append(bt, whole, layout)
    tensors, cache = bt.device()
    cfg0, _, q, k, v, gq, gk, cs, _, _, _, qo = whole["args"]
    done = 0
    for n in (1, 15, 3, 20, 2):
        part = slice(done, done + n)
        cfg = abi.make_kv_append_config(None, k[part], v[part], None, 1, rot_dim=128, n_pos=cfg0.n_pos, rope_layout=cfg0.rope_layout)
        cu, ln = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, n], [done + n]))
        abi.moe_blockkv_append(cfg, cache, None, k[part], v[part], None, gk, cs, None, cu, ln, None)
        done += n
    for a, b in zip(tensors, whole["cache"]):
        assert torch.equal(a, b)


def test_append_sizes_at_every_border():
    """Block maxima at, under and over each scale's limit, elements at the codes' borders, zeros, the largest and the
    smallest sizes."""
    bt = BlockBatch([40, 1], [40, 1], Hkv=8, D=256, seed=6, gk=1.0, gv=2.0 ** -8)
    rng = np.random.default_rng(6)
    s = bo.E4M3_SCALES[rng.integers(0, 126, (41, 8, 16, 1))]
    codes = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0], (41, 8, 16, 16))
    codes[..., 0] = rng.choice([6.0, 6.0 * (1 + 2.0 ** -7), 6.0 * (1 - 2.0 ** -8)], (41, 8, 16))
    x = torch.from_numpy((codes * s * rng.choice([-1.0, 1.0], codes.shape)).reshape(41, 8, 256)).to(torch.bfloat16)
    bt.k.copy_(x)
    bt.v.copy_(x * 2.0 ** -8)
    bt.k[3], bt.v[5] = 0.0, 0.0
    bt.k[7] *= 2.0 ** 40
    bt.v[8] *= 2.0 ** -60
    bt.k[40], bt.v[40] = 3.0e38, 1.0e-38
    check_append(bt, run_append(bt))


def test_append_nonfinite_elements():
    bt = BlockBatch([20, 6], [20, 22], seed=8)
    bt.k[3, 1, 17], bt.v[4, 0, 0] = math.nan, math.nan
    bt.v[21, 0, 5], bt.v[22, 0, 6], bt.k[22, 1, 100] = math.inf, -math.inf, math.inf
    r = run_append(bt)
    assert r["st"] == NONFINITE
    ref = bt.oracle_cache()
    _, written = bo.append(ref, None, values64(bt.k), values64(bt.v), None, None, None, None, bt.cu, bt.kv_len)
    check_cache(bt, r, ref, written)
    for name in "kv":   # one element of each is NaN, and so one block
        assert np.isnan(ref.scale[name]).sum() - np.isnan(bt.oracle_cache().scale[name]).sum() == 1


@pytest.mark.parametrize("fault", ["page_low", "page_high", "table_short", "position", "cu_drop", "cu_high", "len"])
def test_append_faults_are_reported_and_contained(fault):
    bt = BlockBatch([6, 20, 5], [6, 40, 21], seed=9)
    n_pos, positions, skipped = 4096, None, set()
    if fault in ("page_low", "page_high"):
        bt.table[1, 1] = -1 if fault == "page_low" else bt.n_pages
        skipped = {t for t in range(6, 26) if (20 + t - 6) // 16 == 1}
    elif fault == "table_short":
        bt.kv_len[1] += 16 * bt.table.shape[1]
        skipped = set(range(6, 26))
    elif fault == "position":
        positions = np.zeros(bt.T, dtype=np.int32)
        positions[[7, 9]] = [-1, 4096]
        skipped = {7, 9}
    elif fault == "cu_drop":
        bt.cu[2] = 4
        skipped = set(range(4, 31))      # other requests may stay unwritten too
    elif fault == "cu_high":
        bt.cu[3] = bt.T + 7
        skipped = set(range(26, 31))
    elif fault == "len":
        bt.kv_len[1] = 3
        skipped = set(range(6, 26))
    r = run_append(bt, 128, "half", True, n_pos=n_pos, positions=positions)
    assert r["st"] == BOUNDS and abi.moe_get_device_status() == 0
    # the oracle on the requests that are whole, row by row
    ref, written = bt.oracle_cache(), []
    ok = BlockBatch([6, 20, 5], [6, 40, 21], seed=9)
    for b in range(3):
        for i in range(ok.new[b]):
            t, pos = ok.cu[b] + i, ok.total[b] - ok.new[b] + i
            if t in skipped:
                continue
            cs = r["cs"][pos if positions is None else positions[t]]
            for h in range(bt.Hkv):
                for name, row in (("k", bo.key_rows(values64(bt.k)[t, h], r["gk"], cs, "half")), ("v", values64(bt.v)[t, h])):
                    page, slot = ok.table[b, pos // 16], pos % 16
                    ref.codes[name][page, h, slot], ref.scale[name][page, h, slot] = bo.quantise(row, ref.g[name])
                    written.append((name, page, h, slot))
    if fault != "cu_drop":
        check_cache(bt, r, ref, written)
    else:   # only the first four rows are sure
        sure = [w for w in written if w[1] == ok.table[0, 0] and w[3] < 4]
        for i, name in enumerate("kv"):
            scales = bo.decode_e4m3(host(r["cache"][2 + i]))
            assert sure and all(np.array_equal(scales[p, h, s], ref.scale[name][p, h, s]) for n, p, h, s in sure if n == name)
    if fault == "position":
        assert np.all(values64(r["q_out"])[[7, 9]] == 5.0) and np.all(values64(r["q_out"])[8] != 5.0)


def test_rows_of_no_request_are_left_alone():
    """Offsets that begin behind row 0 and end before T (a padded batch)."""
    bt = BlockBatch([3, 30, 9, 6], [3, 33, 50, 6], seed=10)
    r = run_append(bt, 64, "half", True)
    inner = BlockBatch([3, 30, 9, 6], [3, 33, 50, 6], seed=10)
    inner.B, inner.cu, inner.kv_len, inner.table = 2, bt.cu[1:4].copy(), bt.kv_len[1:3].copy(), bt.table[1:3].copy()
    got = run_append(inner, 64, "half", True)
    assert got["st"] == 0
    assert torch.equal(got["q_out"][3:42], r["q_out"][3:42]) and torch.all(got["q_out"][:3] == 5) and torch.all(got["q_out"][42:] == 5)
    ref = inner.oracle_cache()
    _, written = bo.append(ref, None, values64(bt.k), values64(bt.v), None, got["gk"], got["cs"], None, inner.cu, inner.kv_len)
    check_cache(inner, got, ref, written)
    k = torch.full((bt.T, bt.Hkv, bt.D), 9.0, device="cuda")
    abi.moe_blockkv_read(abi.make_blockkv_read_config(k, None, 2), got["args"][1], *inner.lengths(), k, None)
    assert torch.all(k[:3] == 9) and torch.all(k[42:] == 9) and torch.all(k[3:42] != 9)


# ----------------------------------------------------------------- read

def run_read(bt, dtype=torch.bfloat16, wide=0, which="kv", stream=None):
    tensors, cache = bt.device()
    outs = [torch.full((bt.T, bt.Hkv + wide, bt.D), 9.0, dtype=dtype, device="cuda")[:, :bt.Hkv] if n in which else None for n in "kv"]
    torch.cuda.synchronize()
    abi.moe_blockkv_read(abi.make_blockkv_read_config(*outs, batch=bt.B), cache, *bt.lengths(), *outs, stream=stream)
    return outs, abi.moe_get_device_status(stream)


@pytest.mark.parametrize("new,total,kw", [
    ([1], [1], dict()),
    ([1, 1, 1, 1], [15, 16, 17, 300], dict(Hkv=1)),
    ([5, 0, 33, 1], [5, 40, 50, 64], dict(order="nhd", Hkv=5)),
    ([130, 3, 70], [131, 129, 70], dict(D=64, page=128, Hkv=3)),
    ([40, 77], [50, 77], dict(D=256, page=32, Hkv=1)),
    ([100] * 3, [100, 116, 1000], dict(Hkv=8, gk=2.0 ** -9, gv=2.0 ** 40)),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read(new, total, kw, dtype):
    bt = BlockBatch(new, total, seed=sum(total), **kw)
    c = bt.oracle_cache()
    for which, wide, stream in (("kv", 0, None), ("k", 3, torch.cuda.Stream()), ("v", 1, None)):
        outs, st = run_read(bt, dtype, wide, which, stream)
        assert st == 0
        for name, out in zip("kv", outs):
            if out is None:
                continue
            for b in range(bt.B):
                want = np.stack([c.values(name, b, h, bt.total[b])[bt.total[b] - bt.new[b]:] for h in range(bt.Hkv)], 1)
                assert np.array_equal(values64(out)[bt.cu[b]:bt.cu[b + 1]], want)
            if wide:
                assert torch.all(out._base[:, bt.Hkv:] == 9)


@pytest.mark.parametrize("fault", ["page_low", "page_high", "table_short", "cu_drop", "cu_high", "len"])
def test_read_faults(fault):
    bt = BlockBatch([6, 20, 5], [6, 40, 21], seed=9)
    good, _ = run_read(bt)
    rows = range(6, 26)
    if fault in ("page_low", "page_high"):
        bt.table[1, 1] = -2 ** 31 if fault == "page_low" else bt.n_pages
        rows = [t for t in range(6, 26) if (20 + t - 6) // 16 == 1]
    elif fault == "table_short":
        bt.kv_len[1] += 16 * bt.table.shape[1]
    elif fault == "cu_drop":
        bt.cu[2] = 4
        rows = range(4, 31)
    elif fault == "cu_high":
        bt.cu[3] = bt.T + 7
        rows = range(26, 31)
    elif fault == "len":
        bt.kv_len[1] = 19
    out, st = run_read(bt)
    assert st == BOUNDS
    keep = np.array([t not in rows for t in range(bt.T)])
    for a, b in zip(out, good):
        assert np.array_equal(values64(a)[keep], values64(b)[keep])
        if fault != "cu_drop":
            assert np.all(values64(a)[~keep] == 9.0)


def test_nan_scales_are_read_as_nan():
    bt = BlockBatch([4], [20], seed=11)
    bt.scales["k"][bt.table[0, 1], 1, 2, 3] = 0x7F
    (k, v), st = run_read(bt, torch.float32)
    assert st == 0 and torch.isnan(k[2, 1, 48:64]).all() and torch.isnan(k).sum() == 16 and not torch.isnan(v).any()


# ----------------------------------------------------------------- attention

def run_attention(bt, window=0, n_sink=0, max_q_len=0, lse=True, stream=None, q=None, ws=None):
    _, cache = bt.device()
    q = bt.q.cuda() if q is None else q
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda") if lse else None
    cfg = abi.make_paged_attention_config(q, out, bt.B, max_q_len=max_q_len, window=window, n_sink=n_sink)
    need = abi.moe_blockkv_attention_ws_bytes(cfg, cache)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
    torch.cuda.synchronize()
    abi.moe_blockkv_attention(cfg, cache, q, *bt.lengths(), out, ls, ws, stream=stream)
    return out, ls, abi.moe_get_device_status(stream)


def compare(got_o, got_l, ref_o, ref_l, vmax):
    live = ref_l > -math.inf
    assert np.all(got_l[~live] == -math.inf) and np.all(got_o[~live] == 0.0)
    assert np.all(np.abs(got_o - ref_o) <= 2.0 ** -8 * np.abs(ref_o) + 2.0 ** -10 * vmax)
    assert np.all(np.abs(got_l[live] - ref_l[live]) <= 2e-5 * (1 + np.max(np.abs(ref_l[live]), initial=0.0)))


def check_attention(bt, window=0, n_sink=0, **kw):
    out, lse, st = run_attention(bt, window, n_sink, **kw)
    assert st == 0
    ref_o, ref_l = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5, window, n_sink)
    compare(values64(out), values64(lse), ref_o, ref_l, bt.vmax())
    return out, lse


FEW = [
    ([1], [1], dict()),
    ([1], [129], dict(Hq=32, Hkv=4)),
    ([1, 1, 1, 1], [15, 16, 17, 300], dict(Hq=7, Hkv=1)),
    ([1, 1], [65, 63], dict(Hq=2, Hkv=2, order="nhd")),
    ([1, 3, 0, 2], [40, 3, 50, 90], dict(Hq=16, Hkv=1, page=32)),
    ([2, 17], [200, 30], dict(Hq=3, Hkv=3, D=64, page=64)),
    ([1, 5], [130, 128], dict(Hq=40, Hkv=2, D=64, page=128, order="nhd")),
    ([3, 1], [70, 31], dict(Hq=4, Hkv=2, D=256, page=16, gk=2.0 ** -3)),
    ([33], [33], dict(Hq=2, Hkv=1, D=256, page=64)),
    ([150, 40], [150, 230], dict(Hq=8, Hkv=1, page=16)),
    ([70, 1, 129], [90, 77, 129], dict(Hq=4, Hkv=4, page=32, order="nhd")),
    ([40], [300], dict(Hq=14, Hkv=2, D=64, page=16)),
]
# Enough rows, and a page table wide enough, for the tcgen05 kernel; the third and
# the last mix both kernels, the fourth and fifth have equal prompts.
WIDE = dict(extra_width=1024)
MANY = [
    ([64, 130], [900, 130], dict(Hq=16, Hkv=2)),
    ([300], [1500], dict(Hq=7, Hkv=1, D=64, page=64, gk=0.5, gv=4.0)),
    ([1, 100, 0, 3], [700, 2100, 40, 5], dict(Hq=32, Hkv=4, page=32, order="nhd")),
    ([128, 128], [128, 1000], dict(Hq=8, Hkv=8)),
    ([65] * 4, [65, 770, 769, 66], dict(Hq=8, Hkv=8, D=64, page=128)),
    ([1] * 6 + [100] + [1] * 6, [1700] * 6 + [400] + [1700] * 6, dict(Hq=32, Hkv=8, D=64, page=64)),
]


@pytest.mark.parametrize("new,total,kw", FEW)
@pytest.mark.parametrize("hint", [False, True])
def test_attention_few_rows(new, total, kw, hint):
    check_attention(BlockBatch(new, total, seed=sum(total), **kw), max_q_len=max(new) if hint else 0)


@pytest.mark.parametrize("new,total,kw", FEW)
@pytest.mark.parametrize("window", [0, 600])
def test_attention_few_rows_cut(new, total, kw, window):
    """Page tables and windows of over 512 tokens: row tiles may be cut."""
    check_attention(BlockBatch(new, total, seed=sum(total), extra_width=640 // kw.get("page", 16), **kw), window, 2, max_q_len=max(new))


@pytest.mark.parametrize("new,total,kw", [([1, 1], [3000, 500], dict(D=64)), ([2], [1500], dict(D=256, Hkv=1)),
                                          ([4, 3, 1], [1300, 3, 2000], dict(page=64)), ([30], [900], dict(D=128, Hq=2))])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (130, 0), (400, 60), (477, 5), (3, 130)])
def test_attention_few_rows_short_windows(new, total, kw, window, n_sink):
    """Windows of up to 512 tokens in long contexts: row tiles stay whole."""
    check_attention(BlockBatch(new, total, seed=sum(total), **kw), window, n_sink, max_q_len=max(new))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (16, 4), (40, 0), (64, 70), (129, 5), (10 ** 6, 3)])
@pytest.mark.parametrize("new,total,kw", [FEW[2], FEW[5], FEW[9], FEW[7]])
def test_attention_few_rows_window(new, total, kw, window, n_sink):
    check_attention(BlockBatch(new, total, seed=window + n_sink, **kw), window, n_sink, max_q_len=max(new))


@pytest.mark.parametrize("new,total,kw", MANY)
@pytest.mark.parametrize("hint", [False, True])
def test_attention_many_rows(new, total, kw, hint):
    check_attention(BlockBatch(new, total, seed=sum(total), **WIDE, **kw), max_q_len=max(new) if hint else 0)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (130, 4), (900, 300), (10 ** 6, 3)])
@pytest.mark.parametrize("new,total,kw", MANY[:3])
def test_attention_many_rows_window(new, total, kw, window, n_sink):
    check_attention(BlockBatch(new, total, seed=window + n_sink, **WIDE, **kw), window, n_sink, max_q_len=max(new))


@pytest.mark.parametrize("new,total,wide,window", [([1, 4, 60], [200, 300, 260], {}, 50), ([100, 64, 150], [1900, 300, 1260], WIDE, 900)])
def test_attention_evicted_pages(new, total, wide, window):
    """Pages that a window has left behind may be gone from the table, and hold anything."""
    bt = BlockBatch(new, total, Hq=8, Hkv=1, seed=11, **wide)
    ref = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5, window, 4)
    for b in range(bt.B):
        first = bt.total[b] - bt.new[b]
        for pg in range(1, (first - window + 1) // bt.page):
            for n in "kv":
                bt.scales[n][bt.table[b, pg]] = 0x7F
            bt.table[b, pg] = -1
    for hint in (0, max(new)):
        out, lse, st = run_attention(bt, window, 4, max_q_len=hint)
        assert st == 0
        compare(values64(out), values64(lse), *ref, bt.vmax())


@pytest.mark.parametrize("new,kv_len,wide", [([5, 3, 2, 130], [2, 0, -7, 100], {}), ([50, 100, 60, 300], [20, 0, -7, 1100], WIDE)])
def test_attention_rows_that_see_nothing(new, kv_len, wide):
    bt = BlockBatch(new, [max(n, t) for n, t in zip(new, kv_len)], Hq=8, Hkv=1, seed=12, **wide)
    bt.kv_len[:] = kv_len
    for hint in (0, max(new)):
        out, lse = check_attention(bt, max_q_len=hint)
        assert np.all(values64(out)[:new[0] - kv_len[0]] == 0.0)
        assert np.all(values64(lse)[new[0]:sum(new[:3])] == -math.inf)


@pytest.mark.parametrize("new,total,wide", [([2, 1], [70, 40], {}), ([260], [1150], WIDE)])
def test_attention_queries_that_are_not_finite(new, total, wide):
    bt = BlockBatch(new, total, Hq=8, Hkv=2, seed=13, **wide)
    clean_o, clean_l, _ = run_attention(bt, max_q_len=max(new))
    bt.q[1, 3, 5], bt.q[0, 6, 0] = math.nan, math.inf
    out, lse, _ = run_attention(bt, max_q_len=max(new))
    bad = np.zeros((bt.T, 8), dtype=bool)
    bad[1, 3] = bad[0, 6] = True
    assert np.all(np.isnan(values64(out)[bad])) and np.all(np.isnan(values64(lse)[bad]))
    assert np.array_equal(values64(out)[~bad], values64(clean_o)[~bad])
    assert np.array_equal(values64(lse)[~bad], values64(clean_l)[~bad])


@pytest.mark.parametrize("new,total,wide", [([2, 1], [70, 100], {}), ([256], [1140], WIDE)])
def test_attention_extreme_scales_and_scores(new, total, wide):
    """Every scale from 2^-9 to 448, factors far from 1, scores of thousands."""
    bt = BlockBatch(new, total, Hq=8, Hkv=2, seed=14, gk=2.0 ** -30, gv=2.0 ** 30, **wide)
    rng = np.random.default_rng(14)
    for n in "kv":
        s = bt.scales[n]
        bt.scales[n] = np.where(s == 0x7F, s, rng.integers(1, 127, s.shape).astype(np.uint8))
    bt.q.mul_(2.0 ** 25)
    check_attention(bt, max_q_len=max(new))
    bt.q.mul_(2.0 ** 6)
    out, lse, st = run_attention(bt, max_q_len=max(new))
    _, ref_l = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5)
    assert np.max(np.abs(values64(lse) - ref_l)) <= 2e-5 * (1 + np.max(np.abs(ref_l)))


def hide(bt, b, hidden, window=0):
    """fp64 (out, lse) of request b, whose positions `hidden` nobody sees."""
    c, n, total, group = bt.oracle_cache(), int(bt.cu[b + 1] - bt.cu[b]), int(bt.kv_len[b]), bt.Hq // bt.Hkv
    q = values64(bt.q)[bt.cu[b]:bt.cu[b + 1]]
    out, lse = np.zeros_like(q), np.full(q.shape[:2], -math.inf)
    shown = np.array([j not in hidden for j in range(total)])
    for h in range(bt.Hkv):
        K, V = c.values("k", b, h, total), c.values("v", b, h, total)
        for i in range(n):
            see = shown & (np.arange(total) <= total - n + i)
            for hq in range(h * group, (h + 1) * group) if see.any() else ():
                z = bt.D ** -0.5 * (K[see] @ q[i, hq])
                e = np.exp(z - z.max())
                out[i, hq], lse[i, hq] = (e / e.sum()) @ V[see], z.max() + math.log(e.sum())
    return out, lse, bt.vmax()


@pytest.mark.parametrize("bad", [-1, None, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("new,total,pages,kw", [
    ([1, 2], [100, 60], [2, 6], dict(D=64)), ([1, 2], [100, 60], [2, 6], dict(D=128)), ([1, 2], [100, 60], [0, 6], dict(D=256)),
    ([3], [3], [0], {}), ([150], [150], [0, 1], WIDE),
    ([100, 160], [1000, 900], [0, 2, 8, 9, 10, 11, 12, 13, 14, 15, 62], dict(D=64, **WIDE)),
    ([100, 160], [1000, 900], [0, 2, 8, 9, 10, 11, 12, 13, 14, 15, 62], dict(D=128, **WIDE)),
])
def test_attention_pages_out_of_the_cache(new, total, pages, kw, bad):
    """They are reported, and their positions are as if the rows did not see them."""
    bt = BlockBatch(new, total, Hq=8, Hkv=2, seed=31, **kw)
    ref = [hide(bt, b, {j for p in pages for j in range(16 * p, 16 * p + 16)} if b == 0 else set()) for b in range(bt.B)]
    bt.table[0, pages] = bt.n_pages if bad is None else bad
    for hint in (0, max(new)):
        out, lse, st = run_attention(bt, max_q_len=hint)
        assert st == BOUNDS
        for b, (o, l, vmax) in enumerate(ref):
            at = slice(bt.cu[b], bt.cu[b + 1])
            compare(values64(out)[at], values64(lse)[at], o, l, vmax)


@pytest.mark.parametrize("bad", [None, -1, -2 ** 31])
@pytest.mark.parametrize("n,D,Hq", [(2, 64, 4), (2, 128, 4), (2, 256, 4), (5, 128, 3), (3, 64, 5)])
def test_attention_many_requests(n, D, Hq, bad):
    """Pieces of several units and of several requests, most units without masks; pages missing among them."""
    lengths = [1500, 1499, 1281, 1280, 1279, 700, 129, 128, 40, n, 1]
    one = BlockBatch([n], [1500], Hq=Hq, Hkv=1, D=D, seed=32)
    pages = [] if bad is None else [0, 20, 41, 42, 43, 44, 93]
    hidden = {j for p in pages for j in range(16 * p, 16 * p + 16)}
    ref = []
    for length in lengths:
        one.kv_len[0] = length
        ref.append(hide(one, 0, hidden) if pages else
                   (*do.paged_attention(one.oracle_cache(), values64(one.q), one.cu, one.kv_len, D ** -0.5), one.vmax()))
    if pages:
        one.table[0, pages] = bad
    bt, B = one, 60 * len(lengths)
    bt.B, bt.T, bt.q = B, n * B, one.q.repeat(B, 1, 1)
    bt.cu = np.arange(0, n * B + 1, n).astype(np.int32)
    bt.kv_len = np.array(lengths * 60, dtype=np.int32)
    bt.table = np.repeat(one.table, B, 0)
    out, lse, st = run_attention(bt, max_q_len=n)
    assert st == (BOUNDS if pages else 0)
    out, lse = values64(out).reshape(60, len(lengths), n, Hq, D), values64(lse).reshape(60, len(lengths), n, Hq)
    for i, (o, l, vmax) in enumerate(ref):
        for k in range(60):
            compare(out[k, i], lse[k, i], o, l, vmax)


def repeated(bt, times):
    """The batch `times` over, each with pages of its own."""
    n = bt.n_pages
    bt.table = np.concatenate([np.where(bt.table < 0, -1, bt.table + i * n) for i in range(times)]).astype(np.int32)
    bt.cu = np.concatenate([[0]] + [bt.cu[1:] + i * bt.T for i in range(times)]).astype(np.int32)
    bt.new, bt.total, bt.kv_len = bt.new * times, bt.total * times, np.tile(bt.kv_len, times)
    for of in (bt.codes, bt.scales):
        for name in "kv":
            of[name] = np.tile(of[name], (times, 1, 1, 1))
    bt.q, bt.k, bt.v = (x.repeat(times, 1, 1) for x in (bt.q, bt.k, bt.v))
    bt.B, bt.T, bt.n_pages = bt.B * times, bt.T * times, n * times


@pytest.mark.parametrize("new,total,kw,hint", [
    ([1, 2, 0, 1, 1], [40, 16, 9, 130, 1], dict(D=64, Hq=2, Hkv=1), 2),
    ([1, 2, 0, 1, 1], [40, 16, 9, 130, 1], dict(D=128, Hq=2, Hkv=1), 0),
    ([17, 18, 1, 16], [34, 18, 200, 133], dict(D=64, Hq=4, Hkv=1), 18),
    ([17, 17, 17], [34, 17, 140], dict(D=128, Hq=4, Hkv=1), 17),
])
def test_more_requests_than_a_launch_takes(new, total, kw, hint):
    """Slices of 4096 requests, the last one short: of few rows, mixed, and of equal prompts."""
    times = 8200 // len(new)
    bt = BlockBatch(new, total, seed=33, **kw)
    ref_o, ref_l = do.paged_attention(bt.oracle_cache(), values64(bt.q), bt.cu, bt.kv_len, bt.D ** -0.5)
    base = run_append(bt, bt.D), run_read(bt, torch.float32)[0]
    n_pages, vmax = bt.n_pages, bt.vmax()
    repeated(bt, times)
    assert bt.B > 2 * 4096
    out, lse, st = run_attention(bt, max_q_len=hint)
    assert st == 0
    compare(values64(out).reshape(times, *ref_o.shape), values64(lse).reshape(times, *ref_l.shape), ref_o[None].repeat(times, 0),
            ref_l[None].repeat(times, 0), vmax)
    got = run_append(bt, bt.D), run_read(bt, torch.float32)[0]
    assert got[0]["st"] == 0
    assert torch.equal(got[0]["q_out"], base[0]["q_out"].repeat(times, 1, 1))
    for a, b in zip(got[1], base[1]):
        assert torch.equal(a, b.repeat(times, 1, 1))
    for i in range(4):
        a, b = host(got[0]["cache"][i]), host(base[0]["cache"][i])
        assert np.array_equal(a.reshape(times, *b.shape), b[None].repeat(times, 0))


def test_attention_offsets_out_of_order():
    bt = BlockBatch([1, 2], [100, 60], seed=15)
    bt.cu[1] = 9                                          # past T
    out, _, st = run_attention(bt)
    assert st == BOUNDS and np.all(values64(out) == 7.0)
    bt = BlockBatch([300], [1100], Hq=8, Hkv=1, seed=27, **WIDE)
    ref, _, _ = run_attention(bt)
    bt.B, bt.cu, bt.kv_len = 101, np.array([0, 300] * 51, dtype=np.int32), np.full(101, 1100, dtype=np.int32)
    bt.table = np.repeat(bt.table, 101, 0)
    out, _, st = run_attention(bt)
    assert st == BOUNDS
    # every request that names a row has the same result for it, within twice the bound above
    assert np.all(np.abs(values64(out) - values64(ref)) <= 2.0 ** -7 * np.abs(values64(ref)) + 2.0 ** -9 * bt.vmax())


@pytest.mark.parametrize("new,total,kw", [([1, 1, 3, 90], [700, 33, 260, 400], {}), ([1, 256, 3, 90], [1700, 1333, 260, 900], WIDE)])
def test_attention_same_bits_strided_on_another_stream(new, total, kw):
    bt = BlockBatch(new, total, Hq=8, Hkv=2, seed=17, **kw)
    ref, ref_l, st = run_attention(bt, max_q_len=max(new))
    assert st == 0
    for _ in range(3):
        out, lse, _ = run_attention(bt, max_q_len=max(new))
        assert torch.equal(out, ref) and torch.equal(lse, ref_l)
    assert torch.equal(run_attention(bt, max_q_len=max(new), lse=False)[0], ref)
    wide = torch.zeros(bt.T, bt.Hq + 3, bt.D, dtype=torch.bfloat16, device="cuda")
    wide[:, :bt.Hq] = bt.q.cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, lse, st = run_attention(bt, max_q_len=max(new), stream=s, q=wide[:, :bt.Hq])
    s.synchronize()
    assert st == 0 and torch.equal(out, ref) and torch.equal(lse, ref_l)


def test_attention_two_calls_at_once():
    """Each with its own workspace, on two streams; one after the other they may share it."""
    a, b = (BlockBatch([2, 70, 1], [900, 800, 700], Hq=8, Hkv=2, seed=s, **WIDE) for s in (40, 41))
    ref = [run_attention(x, max_q_len=70)[:2] for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = []
    for x, s in zip((a, b), streams):
        _, cache = x.device()
        q, lengths = x.q.cuda(), x.lengths()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        cfg = abi.make_paged_attention_config(q, out, x.B, max_q_len=70)
        ws = torch.empty(abi.moe_blockkv_attention_ws_bytes(cfg, cache), dtype=torch.uint8, device="cuda")
        calls.append((cfg, cache, q, *lengths, out, lse, ws, s))
    torch.cuda.synchronize()
    for _ in range(5):
        for c in calls:
            abi.moe_blockkv_attention(*c)
    torch.cuda.synchronize()
    for c, r in zip(calls, ref):
        assert torch.equal(c[5], r[0]) and torch.equal(c[6], r[1])
    for c, r in zip(calls, ref):
        abi.moe_blockkv_attention(*c[:7], calls[0][7])
        assert torch.equal(c[5], r[0]) and torch.equal(c[6], r[1])


def test_attention_weights_of_many_small_ones():
    """65535 keys 2^-20 of the first one's weight: together 1/16 of the sum; the first has no value."""
    n, D = 65536, 128
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16)
    q[0, 0, 0] = 1.0
    k = torch.zeros(n // 128, 1, 128, D // 2, dtype=torch.uint8)
    k[0, 0, 0, 0] = 7                                     # 6: the first key's score, in units of g
    v = torch.full((n // 128, 1, 128, D // 2), 0x22, dtype=torch.uint8)   # 1.0
    v[0, 0, 0] = 0
    one = torch.full((n // 128, 1, 128, D // 16), 0x38, dtype=torch.uint8)
    table = torch.arange(n // 128, dtype=torch.int32).view(1, -1)
    dev = [t.cuda() for t in (k, v, one, one.clone(), table)]
    cache = abi.make_blockkv_cache(*dev)
    out = torch.empty(1, 1, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 1, device="cuda")
    cfg = abi.make_paged_attention_config(q, out, 1, max_q_len=1, sm_scale=20 * math.log(2) / 6)
    ws = torch.empty(abi.moe_blockkv_attention_ws_bytes(cfg, cache), dtype=torch.uint8, device="cuda")
    cu, ln = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 1], [n]))
    abi.moe_blockkv_attention(cfg, cache, q.cuda(), cu, ln, out, lse, ws)
    small = (n - 1) * 2.0 ** -20
    want = small / (1 + small)
    assert abi.moe_get_device_status() == 0
    # weights of 2^-20 of the largest keep their 11 bits: 2^-11, and one bf16 rounding
    assert torch.all((out.double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -11))
    assert abs(lse.item() - (20 * math.log(2) + math.log1p(small))) <= 2e-5 * 15


def test_past_32_bit_offsets():
    """A cache of over 4 GB of codes: byte offsets need 64 bits, in all three calls."""
    D, page, n_pages = 256, 128, 280_000                  # 4.6 GB of key codes, 0.57 of scales, the same of values
    k, v = (torch.zeros(n_pages, 1, page, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pages, 1, page, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32, device="cuda")
    cache = abi.make_blockkv_cache(k, v, ks, vs, table)
    g = torch.Generator().manual_seed(19)
    n = 300
    kn, vn = (torch.randn(n, 1, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(n, 4, D, generator=g).to(torch.bfloat16).cuda()
    qo, out = torch.empty_like(q), torch.empty_like(q)
    cu, ln = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, n], [n]))
    abi.moe_blockkv_append(abi.make_kv_append_config(q, kn, vn, qo, 1), cache, q, kn, vn, None, None, None, None, cu, ln, qo)
    K, V = (torch.empty(n, 1, D, device="cuda") for _ in range(2))
    abi.moe_blockkv_read(abi.make_blockkv_read_config(K, V, 1), cache, cu, ln, K, V)
    cfg = abi.make_paged_attention_config(qo, out, 1, max_q_len=n)
    ws = torch.empty(abi.moe_blockkv_attention_ws_bytes(cfg, cache), dtype=torch.uint8, device="cuda")
    abi.moe_blockkv_attention(cfg, cache, qo, cu, ln, out, None, ws)
    assert abi.moe_get_device_status() == 0
    for got, x in ((K, kn), (V, vn)):
        for t in (0, 127, 128, 299):
            codes, scales = bo.quantise(x[t, 0].float().cpu().numpy(), 1.0)
            assert np.array_equal(got[t, 0].double().cpu().numpy(), codes * np.repeat(scales, 16))
    K, V = K[:, 0].double(), V[:, 0].double()
    z = torch.einsum("thd,jd->htj", q.double(), K) * D ** -0.5
    z = z.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -math.inf)
    ref = torch.einsum("htj,jd->thd", torch.softmax(z, -1), V)
    assert torch.all((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * V.abs().max())


# ----------------------------------------------------------------- together

def test_append_attend_and_read_in_a_graph():
    """All three calls captured on a side stream and replayed on new inputs and lengths."""
    bt = BlockBatch([1, 1, 1], [20, 1, 50], Hq=8, Hkv=2, seed=18)
    tensors, cache = bt.device()
    q, k, v = bt.q.cuda(), bt.k.cuda(), bt.v.cuda()
    qo, out = torch.empty_like(q), torch.empty_like(q)
    rows = torch.empty_like(k), torch.empty_like(k)
    cu, kv_len = bt.lengths()
    cs = torch.from_numpy(angles(64, 128)).cuda()
    ca = abi.make_kv_append_config(q, k, v, qo, bt.B, rot_dim=128, n_pos=64)
    cp = abi.make_paged_attention_config(qo, out, bt.B, max_q_len=1)
    cr = abi.make_blockkv_read_config(*rows, bt.B)
    ws = torch.empty(abi.moe_blockkv_attention_ws_bytes(cp, cache), dtype=torch.uint8, device="cuda")

    def step():
        abi.moe_blockkv_append(ca, cache, q, k, v, None, None, cs, None, cu, kv_len, qo)
        abi.moe_blockkv_attention(cp, cache, qo, cu, kv_len, out, None, ws)
        abi.moe_blockkv_read(cr, cache, cu, kv_len, *rows)

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
    saved = [x.clone() for x in tensors]
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (out, *rows, *tensors)]
    for x, y in zip(tensors, saved):
        x.copy_(y)
    step()
    assert abi.moe_get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, (out, *rows, *tensors)))
