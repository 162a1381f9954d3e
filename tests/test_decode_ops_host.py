"""Host-side checks of the decoder-step operators: refusals before anything is
launched (no GPU needed), the binding's shape checks, and pins of the fp64
oracle that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import top_routed_expert_gb300 as moe
from oracle import decode_oracle as do
from oracle import qk_rope_oracle as qr
from top_routed_expert_gb300 import abi

OK, ODD = 0x10000, 0x10002     # never dereferenced: validation comes first


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return abi.load()


# ----------------------------------------------------------------- refusals

def route_cfg(**kw):
    base = dict(T=4, n_experts=128, top_k=6, n_groups=8, top_groups=4, group_rank=2, score=1, logit_dtype=0,
                renormalise=1, scale=1.0, logit_stride=128)
    base.update(kw)
    return abi.moe_route_scores_config_t(**base)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(n_experts=0), dict(n_experts=257, n_groups=1, top_groups=1, logit_stride=257), dict(top_k=0),
    dict(top_k=17), dict(n_groups=0), dict(n_groups=3), dict(n_groups=64), dict(top_groups=0), dict(top_groups=9),
    dict(n_groups=32, top_groups=1, top_k=5), dict(group_rank=0), dict(group_rank=3), dict(score=2),
    dict(logit_dtype=abi.MOE_E4M3), dict(renormalise=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
    dict(scale=math.nan), dict(logit_stride=127),
])
def test_route_scores_refuses(lib, bad):
    assert lib.moe_route_scores(route_cfg(**bad), OK, None, OK, OK, None) == 1


def test_route_scores_refuses_pointers(lib):
    assert lib.moe_route_scores(None, OK, None, OK, OK, None) == 1
    for args in ((None, None, OK, OK), (OK, None, None, OK), (OK, None, OK, None), (ODD, None, OK, OK),
                 (OK, ODD, OK, OK), (OK, None, ODD, OK), (OK, None, OK, ODD)):
        assert lib.moe_route_scores(route_cfg(), *args, None) == 1
    assert lib.moe_route_scores(route_cfg(logit_dtype=abi.MOE_BF16), 0x10001, None, OK, OK, None) == 1
    assert lib.moe_route_scores(route_cfg(T=0), None, None, None, None, None) == 0


def cache(**kw):
    base = dict(k=OK, v=OK, k_scale=OK, v_scale=OK, page_table=OK, n_pages=9, page_size=16, n_kv_heads=4, head_dim=128,
                max_pages=5, page_stride=8192, head_stride=2048, token_stride=128)
    base.update(kw)
    return abi.moe_kv_cache_t(**base)


BAD_CACHES = [
    dict(n_pages=0), dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(n_kv_heads=0),
    dict(n_kv_heads=1025), dict(head_dim=96), dict(head_dim=512), dict(max_pages=0), dict(max_pages=(1 << 26) + 1),
    dict(page_stride=0), dict(head_stride=-2048), dict(token_stride=64), dict(token_stride=136),
]
BAD_CACHE_POINTERS = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(page_table=None),
                      dict(k=0x10008), dict(v=0x10008), dict(k_scale=ODD), dict(v_scale=ODD), dict(page_table=ODD)]


def append_cfg(**kw):
    base = dict(T=3, batch=2, n_q_heads=32, rot_dim=128, rope_layout=0, n_pos=64, eps=1e-6, q_stride=4096,
                k_stride=512, v_stride=512, q_out_stride=4096)
    base.update(kw)
    return abi.moe_kv_append_config_t(**base)


def append(lib, cfg=None, c=None, q=OK, k=OK, v=OK, gq=OK, gk=OK, cs=OK, pos=None, cu=OK, ln=OK, qo=OK):
    return lib.moe_kv_append(cfg or append_cfg(), c or cache(), q, k, v, gq, gk, cs, pos, cu, ln, qo, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(batch=0), dict(batch=4097), dict(n_q_heads=0), dict(n_q_heads=4097), dict(rot_dim=-8),
    dict(rot_dim=12), dict(rot_dim=136), dict(rope_layout=2), dict(n_pos=0), dict(eps=0.0), dict(eps=math.nan),
    dict(eps=math.inf), dict(q_stride=4088), dict(q_stride=4100), dict(k_stride=504), dict(v_stride=513),
    dict(q_out_stride=0),
])
def test_kv_append_refuses(lib, bad):
    assert append(lib, cfg=append_cfg(**bad)) == 1


@pytest.mark.parametrize("bad", BAD_CACHES + BAD_CACHE_POINTERS)
def test_kv_append_refuses_caches(lib, bad):
    assert append(lib, c=cache(**bad)) == 1


def test_kv_append_refuses_pointers(lib):
    for name in ("k", "v", "cu", "ln", "qo", "cs"):
        assert append(lib, **{name: None}) == 1, name
    for name in ("q", "k", "v", "gq", "gk", "cs", "qo"):
        assert append(lib, **{name: 0x10008}) == 1, name
    for name in ("pos", "cu", "ln"):
        assert append(lib, **{name: ODD}) == 1, name
    assert lib.moe_kv_append(None, cache(), *[OK] * 10, None) == 1
    assert lib.moe_kv_append(append_cfg(), None, *[OK] * 10, None) == 1
    assert append(lib, cfg=append_cfg(T=0), q=None, k=None, v=None, cu=None, ln=None) == 0


def attention_cfg(**kw):
    base = dict(T=3, batch=2, n_q_heads=32, max_q_len=2, window=0, n_sink=0, sm_scale=0.1, q_stride=4096,
                out_stride=4096)
    base.update(kw)
    return abi.moe_paged_attention_config_t(**base)


def attend(lib, cfg=None, c=None, q=OK, cu=OK, ln=OK, out=OK, lse=OK, ws=OK, n=1 << 40):
    return lib.moe_paged_attention(cfg or attention_cfg(), c or cache(), q, cu, ln, out, lse, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(batch=0), dict(batch=4097), dict(n_q_heads=0), dict(n_q_heads=30), dict(n_q_heads=1028),
    dict(max_q_len=-1), dict(window=-1), dict(window=(1 << 30) + 1), dict(n_sink=-1), dict(n_sink=(1 << 30) + 1),
    dict(sm_scale=0.0), dict(sm_scale=math.inf), dict(sm_scale=math.nan), dict(q_stride=4088), dict(out_stride=4097),
    dict(T=1 << 28, n_q_heads=32),
])
def test_attention_refuses(lib, bad):
    c = attention_cfg(**bad)
    assert lib.moe_paged_attention_ws_bytes(c, cache()) == 0
    assert attend(lib, cfg=c) == 1


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_attention_refuses_caches(lib, bad):
    assert lib.moe_paged_attention_ws_bytes(attention_cfg(), cache(**bad)) == 0
    assert attend(lib, c=cache(**bad)) == 1


def test_attention_refuses_pointers_and_workspaces(lib):
    for bad in BAD_CACHE_POINTERS:
        assert attend(lib, c=cache(**bad)) == 1
    for name in ("q", "cu", "ln", "out"):
        assert attend(lib, **{name: None}) == 1, name
    for name in ("q", "out"):
        assert attend(lib, **{name: 0x10008}) == 1, name
    for name in ("cu", "ln", "lse"):
        assert attend(lib, **{name: ODD}) == 1, name
    need = lib.moe_paged_attention_ws_bytes(attention_cfg(), cache())
    assert need > 0
    assert attend(lib, ws=None) == 3 and attend(lib, n=need - 1) == 3
    assert attend(lib, ws=0x10010) == 1
    assert attend(lib, cfg=attention_cfg(T=0), q=None, out=None, ws=None, n=0) == 0


def test_attention_workspace_of_the_largest_call_serves_all(lib):
    def need(T, batch, hint):
        return lib.moe_paged_attention_ws_bytes(attention_cfg(T=T, batch=batch, max_q_len=hint), cache(n_kv_heads=2))

    for batch in (1, 3, 200):
        sizes = [need(T, batch, 0) for T in (1, 7, 64, 300, 1024, 5000, 40000)]
        assert sizes[0] > 0 and sizes == sorted(sizes)
        for T in (7, 300, 40000):
            by_hint = [need(T, batch, h) for h in sorted((1, 6, 7, 100, T // 3, T)) + [0]]
            assert by_hint == sorted(by_hint)


def test_binding_checks_tensors():
    codes = torch.zeros(3, 2, 16, 64, dtype=torch.uint8)
    sc, table = torch.ones(3, 2), torch.zeros(1, 2, dtype=torch.int32)
    c = abi.make_kv_cache(codes, codes, sc, sc, table)
    assert (c.n_pages, c.page_size, c.n_kv_heads, c.head_dim, c.max_pages) == (3, 16, 2, 64, 2)
    assert (c.page_stride, c.head_stride, c.token_stride) == (2048, 1024, 64)
    nhd = torch.zeros(3, 16, 2, 64, dtype=torch.uint8).transpose(1, 2)
    c = abi.make_kv_cache(nhd, nhd, sc, sc, table)
    assert (c.page_stride, c.head_stride, c.token_stride) == (2048, 64, 128)
    for bad in ((codes, nhd, sc, sc, table), (codes.float(), codes.float(), sc, sc, table),
                (codes, codes, sc.double(), sc, table), (codes, codes, sc, sc[:2], table),
                (codes, codes, sc, sc, table.long()), (codes.transpose(2, 3), codes.transpose(2, 3), sc, sc, table)):
        with pytest.raises(ValueError):
            abi.make_kv_cache(*bad)
    q = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    assert abi.make_paged_attention_config(q, q, 2).sm_scale == 0.125
    wide = torch.zeros(4, 9, 64, dtype=torch.bfloat16)[:, :6]
    assert abi.make_paged_attention_config(wide, q, 2).q_stride == 576
    for bad in (q.float(), q.transpose(0, 1), torch.zeros(4, 12, 64, dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(ValueError):
            abi.make_paged_attention_config(bad, bad, 2)


# ----------------------------------------------------------------- oracle pins

def test_oracle_route_matches_closed_forms():
    # two experts, sigmoid: logits ln 3 and 0 have scores 3/4 and 1/2
    ids, w, _ = do.route_scores([[0.0, math.log(3.0)]], None, 2, kind="sigmoid")
    assert ids.tolist() == [[1, 0]] and np.allclose(w, [[0.6, 0.4]])
    _, w, _ = do.route_scores([[0.0, math.log(3.0)]], None, 2, kind="sigmoid", renormalise=False, scale=2.0)
    assert np.allclose(w, [[1.5, 1.0]])
    # a bias moves the choice, not the weight
    ids, w, _ = do.route_scores([[0.0, math.log(3.0)]], [0.3, 0.0], 1, kind="sigmoid", renormalise=False)
    assert ids.tolist() == [[0]] and np.allclose(w, [[0.5]])
    # groups by one value and by two: {0.9, 0.1} against {0.6, 0.5}
    L = [[math.log(9.0), math.log(1 / 9), math.log(1.5), 0.0]]
    assert do.route_scores(L, None, 1, 2, 1, 1, "sigmoid")[0].tolist() == [[0]]
    assert do.route_scores(L, None, 1, 2, 1, 2, "sigmoid")[0].tolist() == [[2]]


def test_oracle_route_matches_torch_and_the_layer_oracle():
    import oracle
    rng = np.random.default_rng(1)
    L = rng.standard_normal((40, 64))
    ids, w, _ = do.route_scores(L, None, 6)
    assert np.array_equal(ids, oracle.topk_ids(L, 6)) and np.allclose(w, oracle.gates(L, ids))
    p, i = torch.softmax(torch.from_numpy(L), 1).topk(6, 1)
    assert np.array_equal(ids, i.numpy()) and np.allclose(w, (p / p.sum(1, keepdim=True)).numpy())


def test_oracle_append_matches_torch():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 64)) * 3
    codes = np.zeros((2, 3, 16, 64), dtype=np.uint8)
    c = do.Cache(codes, codes, np.ones((2, 3)), np.ones((2, 3)), [[1, 0]])
    do.kv_append(c, None, x, x, None, None, None, None, [0, 5], [5])
    for h in range(3):
        s = c.scale["k"][1, h]
        amax = np.abs(x[:, h]).max()
        assert amax <= 448 * s and amax > 224 * s
        want = torch.from_numpy(x[:, h] / s).float().to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(c.codes["k"][1, h, :5], want)
    # a larger token in the same page rounds the earlier codes to its scale
    was = c.codes["k"][1, 0, :5] * c.scale["k"][1, 0]
    do.kv_append(c, None, 64 * x[:1], x[:1], None, None, None, None, [0, 1], [6])
    assert c.scale["k"][1, 0] > 2 ** -6
    assert np.allclose(c.codes["k"][1, 0, :5] * c.scale["k"][1, 0], was, atol=2.0 ** -10 * c.scale["k"][1, 0])


def test_oracle_rotation():
    rng = np.random.default_rng(3)
    y = rng.standard_normal((4, 64))
    cs = qr.rope_table(50, 64)[17]
    gamma = rng.uniform(0.5, 1.5, 64)
    want = qr.rope_rotate_half(qr.rms_norm(y, gamma, 1e-6), cs[:, 0], cs[:, 1])
    assert np.allclose(do.norm_rotate(y, gamma, cs, "half", 1e-6), want)
    # the interleaved layout is the half layout of the permuted head
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    inter = do.norm_rotate(y, None, cs, "interleaved", 1e-6)
    assert np.allclose(inter[:, perm], do.norm_rotate(y[:, perm], None, cs, "half", 1e-6))
    # part of the head: the rest stays
    part = do.norm_rotate(y, None, cs[:8], "half", 1e-6)
    assert np.array_equal(part[:, 16:], y[:, 16:]) and not np.allclose(part[:, :16], y[:, :16])


def test_oracle_attention_matches_torch():
    rng = np.random.default_rng(4)
    codes = torch.from_numpy(rng.standard_normal((6, 2, 16, 64)) * 50).float().to(torch.float8_e4m3fn)
    scale = 2.0 ** rng.integers(-7, -4, (6, 2))
    c = do.Cache(codes.view(torch.uint8).numpy(), codes.flip(0).view(torch.uint8).numpy(), scale, scale[::-1],
                 [[4, 1, 0], [2, 5, 3]])
    q = rng.standard_normal((7, 4, 64))
    cu, total = [0, 3, 7], [40, 21]
    for window, sink in ((0, 0), (8, 0), (8, 2)):
        out, lse = do.paged_attention(c, q, cu, total, 0.125, window, sink)
        for b in range(2):
            n = cu[b + 1] - cu[b]
            p = torch.arange(total[b] - n, total[b])[:, None]
            j = torch.arange(total[b])[None]
            see = (j <= p) & ((j > p - window) | (j < sink) | (window == 0))
            for h in range(4):
                K, V = (torch.from_numpy(c.values(x, b, h // 2, total[b])) for x in ("k", "v"))
                qt = torch.from_numpy(q[cu[b]:cu[b + 1], h])
                want = torch.nn.functional.scaled_dot_product_attention(qt[None], K[None], V[None], see[None], scale=0.125)
                assert np.allclose(out[cu[b]:cu[b + 1], h], want[0].numpy())
                z = (0.125 * qt @ K.T).masked_fill(~see, -math.inf)
                assert np.allclose(lse[cu[b]:cu[b + 1], h], torch.logsumexp(z, 1).numpy())


@pytest.mark.parametrize("wrong", ["causal", "window", "sink", "group", "scale"])
def test_a_mistake_in_the_attention_oracle_is_seen(monkeypatch, wrong):
    """Plausible mistakes change what the pin above compares."""
    def mistaken(c, q, cu, total, sm_scale, window=0, n_sink=0):
        if wrong == "causal":
            total = [t + 0 for t in total]
            cu, q = cu, q[::-1].copy()
        if wrong == "window":
            window += 1 if window else 0
        if wrong == "sink":
            n_sink = 0
        if wrong == "group":
            q = q[:, [0, 2, 1, 3]]
        if wrong == "scale":
            sm_scale *= 1.01
        return real(c, q, cu, total, sm_scale, window, n_sink)
    real = do.paged_attention
    monkeypatch.setattr(do, "paged_attention", mistaken)
    with pytest.raises(AssertionError):
        test_oracle_attention_matches_torch()
