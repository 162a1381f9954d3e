"""Host-side checks of the 4-bit cache's operators and of the addition with the
norm: the C ABI's refusals before anything is launched, and the binding's
checks of what a call names (no GPU needed)."""
import math

import pytest
import torch

import top_routed_expert_gb300 as moe
from tests.test_decode_binding_host import (B, BF16, D, F32, HKV, HQ, I32, PAGE, T, elsewhere, lib as fake_lib,  # noqa: F401
                                            short)
from tests.test_decode_ops_host import append_cfg, attention_cfg
from top_routed_expert_gb300 import abi

OK, ODD = 0x10000, 0x10002     # never dereferenced: validation comes first


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return abi.load()


# ----------------------------------------------------------------- the C ABI

def cache(**kw):
    base = dict(k=OK, v=OK, k_scale=OK, v_scale=OK, page_table=OK, n_pages=9, page_size=16, n_kv_heads=4, head_dim=128,
                max_pages=5, k_gscale=1.0, v_gscale=0.5, page_stride=4096, head_stride=1024, token_stride=64,
                scale_page_stride=512, scale_head_stride=128, scale_token_stride=8)
    base.update(kw)
    return abi.moe_blockkv_cache_t(**base)


BAD_CACHES = [
    dict(n_pages=0), dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(n_kv_heads=0), dict(n_kv_heads=1025),
    dict(head_dim=96), dict(head_dim=512), dict(max_pages=0), dict(max_pages=(1 << 26) + 1), dict(page_stride=0),
    dict(head_stride=-1024), dict(token_stride=48), dict(token_stride=72), dict(scale_page_stride=0),
    dict(scale_head_stride=-128), dict(scale_token_stride=4), dict(scale_token_stride=12), dict(k_gscale=0.0),
    dict(k_gscale=3.0), dict(k_gscale=-1.0), dict(v_gscale=math.nan), dict(v_gscale=math.inf), dict(v_gscale=2.0 ** 61),
    dict(k_gscale=2.0 ** -61), dict(n_pages=1 << 20, page_stride=1 << 16), dict(n_pages=1 << 20, scale_page_stride=1 << 15),
]
BAD_POINTERS = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(page_table=None), dict(k=0x10008),
                dict(v=0x10008), dict(k_scale=0x10004), dict(v_scale=ODD), dict(page_table=ODD)]


def append(lib, cfg=None, c=None, q=OK, k=OK, v=OK, gq=OK, gk=OK, cs=OK, pos=None, cu=OK, ln=OK, qo=OK):
    return lib.moe_blockkv_append(cfg or append_cfg(), c or cache(), q, k, v, gq, gk, cs, pos, cu, ln, qo, None)


def attend(lib, cfg=None, c=None, q=OK, cu=OK, ln=OK, out=OK, lse=OK, ws=OK, n=1 << 40):
    return lib.moe_blockkv_attention(cfg or attention_cfg(), c or cache(), q, cu, ln, out, lse, ws, n, None)


def read_cfg(**kw):
    base = dict(T=3, batch=2, out_dtype=abi.MOE_BF16, k_stride=512, v_stride=512)
    base.update(kw)
    return abi.moe_blockkv_read_config_t(**base)


def read(lib, cfg=None, c=None, cu=OK, ln=OK, k=OK, v=OK):
    return lib.moe_blockkv_read(cfg or read_cfg(), c or cache(), cu, ln, k, v, None)


@pytest.mark.parametrize("bad", BAD_CACHES + BAD_POINTERS)
def test_caches_refused(lib, bad):
    c = cache(**bad)
    assert append(lib, c=c) == attend(lib, c=c) == read(lib, c=c) == 1
    if bad in BAD_CACHES:
        assert lib.moe_blockkv_attention_ws_bytes(attention_cfg(), c) == 0


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(batch=0), dict(batch=2 ** 20 + 1), dict(n_q_heads=0), dict(rot_dim=12), dict(rot_dim=136), dict(rope_layout=2),
    dict(n_pos=0), dict(eps=0.0), dict(eps=math.nan), dict(q_stride=4088), dict(k_stride=504), dict(v_stride=513),
    dict(q_out_stride=0),
])
def test_append_refuses(lib, bad):
    assert append(lib, cfg=append_cfg(**bad)) == 1


def test_append_refuses_pointers(lib):
    for name in ("k", "v", "cu", "ln", "qo", "cs"):
        assert append(lib, **{name: None}) == 1, name
    for name in ("q", "k", "v", "gq", "gk", "cs", "qo"):
        assert append(lib, **{name: 0x10008}) == 1, name
    for name in ("pos", "cu", "ln"):
        assert append(lib, **{name: ODD}) == 1, name
    assert lib.moe_blockkv_append(None, cache(), *[OK] * 10, None) == 1
    assert lib.moe_blockkv_append(append_cfg(), None, *[OK] * 10, None) == 1
    assert append(lib, cfg=append_cfg(T=0), q=None, k=None, v=None, cu=None, ln=None) == 0


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(batch=0), dict(batch=2 ** 20 + 1), dict(n_q_heads=30), dict(n_q_heads=1028), dict(max_q_len=-1), dict(window=-1),
    dict(n_sink=-1), dict(sm_scale=0.0), dict(sm_scale=math.inf), dict(q_stride=4088), dict(out_stride=4097),
    dict(T=1 << 28, n_q_heads=32),
])
def test_attention_refuses(lib, bad):
    c = attention_cfg(**bad)
    assert lib.moe_blockkv_attention_ws_bytes(c, cache()) == 0
    assert attend(lib, cfg=c) == 1


def test_attention_refuses_pointers_and_workspaces(lib):
    for name in ("q", "cu", "ln", "out"):
        assert attend(lib, **{name: None}) == 1, name
    for name, bad in (("q", 0x10008), ("out", 0x10008), ("cu", ODD), ("ln", ODD), ("lse", ODD)):
        assert attend(lib, **{name: bad}) == 1, name
    need = lib.moe_blockkv_attention_ws_bytes(attention_cfg(), cache())
    assert need > 0
    assert attend(lib, n=need - 1) == 3 and attend(lib, ws=None) == 3 and attend(lib, ws=OK + 128) == 1
    assert lib.moe_blockkv_attention(None, cache(), *[OK] * 6, 1 << 40, None) == 1
    assert lib.moe_blockkv_attention(attention_cfg(), None, *[OK] * 6, 1 << 40, None) == 1
    assert lib.moe_blockkv_attention_ws_bytes(None, cache()) == lib.moe_blockkv_attention_ws_bytes(attention_cfg(), None) == 0
    assert attend(lib, cfg=attention_cfg(T=0), q=None, out=None) == 0


@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_workspace_never_shrinks(lib, head_dim):
    c = cache(head_dim=head_dim, max_pages=4096, page_stride=1 << 16, scale_page_stride=1 << 12, token_stride=128,
              scale_token_stride=16)
    size = lambda **kw: lib.moe_blockkv_attention_ws_bytes(attention_cfg(q_stride=32 * 256, out_stride=32 * 256, **kw), c)
    last = 0
    for T in (1, 7, 64, 500, 4096, 70000):
        for batch, m in ((1, 1), (1, 5), (40, 5), (40, 300), (4096, 300), (4096, 0)):
            assert size(T=T, batch=batch, max_q_len=m) >= size(T=T, batch=1, max_q_len=1)
        assert size(T=T, batch=64, max_q_len=0) >= last
        last = size(T=T, batch=64, max_q_len=0)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(batch=0), dict(batch=2 ** 20 + 1), dict(out_dtype=abi.MOE_E4M3), dict(k_stride=504),
                                 dict(v_stride=504), dict(k_stride=516)])
def test_read_refuses(lib, bad):
    assert read(lib, cfg=read_cfg(**bad)) == 1


def test_read_refuses_pointers(lib):
    for name, bad in (("cu", None), ("ln", None), ("cu", ODD), ("ln", ODD), ("k", 0x10008), ("v", 0x10008)):
        assert read(lib, **{name: bad}) == 1, name
    assert lib.moe_blockkv_read(None, cache(), OK, OK, OK, OK, None) == 1
    assert lib.moe_blockkv_read(read_cfg(), None, OK, OK, OK, OK, None) == 1
    assert read(lib, cfg=read_cfg(T=0)) == 0
    assert read(lib, k=None, v=None) == 0


def norm_cfg(**kw):
    base = dict(T=3, d=512, x_dtype=1, res_dtype=1, out_dtype=1, group=128, eps=1e-6, x_stride=512, res_stride=512,
                sum_stride=512, out_stride=512)
    base.update(kw)
    return abi.moe_add_norm_config_t(**base)


def norm(lib, cfg=None, x=OK, res=OK, gamma=OK, out=OK, out8=OK, scale=OK, total=OK):
    return lib.moe_add_rms_norm(cfg or norm_cfg(), x, res, gamma, out, out8, scale, total, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(d=0), dict(d=516), dict(d=16392, x_stride=1 << 15, res_stride=1 << 15, sum_stride=1 << 15, out_stride=1 << 15),
    dict(x_dtype=2), dict(res_dtype=3), dict(out_dtype=2), dict(group=8), dict(group=512), dict(group=-1), dict(group=48),
    dict(d=320, group=128), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf), dict(eps=-1.0), dict(x_stride=504),
    dict(res_stride=516), dict(sum_stride=0), dict(out_stride=511),
])
def test_norm_refuses(lib, bad):
    assert norm(lib, cfg=norm_cfg(**bad)) == 1


def test_norm_refuses_pointers(lib):
    for name in ("x", "gamma", "scale"):
        assert norm(lib, **{name: None}) == 1, name
    for name in ("x", "res", "gamma", "out", "total"):
        assert norm(lib, **{name: 0x10008}) == 1, name
    assert norm(lib, out8=0x10004) == norm(lib, scale=ODD) == 1
    assert norm(lib, out=None, out8=None) == 1
    assert norm(lib, res=None) == 1                       # a sum without a residual
    assert lib.moe_add_rms_norm(None, *[OK] * 7, None) == 1
    assert norm(lib, cfg=norm_cfg(T=0), x=None, gamma=None) == 0


# ----------------------------------------------------------------- the binding

def cache_tensors():
    codes, scales = torch.zeros(9, HKV, PAGE, D // 2, dtype=torch.uint8), torch.zeros(9, HKV, PAGE, D // 16, dtype=torch.uint8)
    return dict(k=codes, v=codes.clone(), k_scale=scales, v_scale=scales.clone(), page_table=torch.zeros(B, 4, dtype=I32))


def append_args(**kw):
    q, k = torch.zeros(T, HQ, D, dtype=BF16), torch.zeros(T, HKV, D, dtype=BF16)
    a = dict(q=q, k=k, v=k.clone(), gamma_q=torch.ones(D), gamma_k=torch.ones(D), cos_sin=torch.zeros(50, D // 2, 2),
             positions=torch.zeros(T, dtype=I32), cu=torch.zeros(B + 1, dtype=I32), kv_len=torch.zeros(B, dtype=I32),
             q_out=torch.zeros_like(q), cache=abi.make_blockkv_cache(**cache_tensors()))
    a["cfg"] = abi.make_kv_append_config(a["q"], a["k"], a["v"], a["q_out"], B, rot_dim=D, n_pos=50)
    a.update(kw)
    return a


def attend_args(**kw):
    q = torch.zeros(T, HQ, D, dtype=BF16)
    a = dict(q=q, cu=torch.zeros(B + 1, dtype=I32), kv_len=torch.zeros(B, dtype=I32), out=torch.zeros_like(q),
             lse=torch.zeros(T, HQ), ws=torch.zeros(64, dtype=torch.uint8), cache=abi.make_blockkv_cache(**cache_tensors()))
    a["cfg"] = abi.make_paged_attention_config(a["q"], a["out"], B)
    a.update(kw)
    return a


def read_args(**kw):
    rows = torch.zeros(T, HKV, D, dtype=kw.pop("dtype", BF16))
    a = dict(cu=torch.zeros(B + 1, dtype=I32), kv_len=torch.zeros(B, dtype=I32), k_out=rows, v_out=rows.clone(),
             cache=abi.make_blockkv_cache(**cache_tensors()))
    a["cfg"] = abi.make_blockkv_read_config(a["k_out"], a["v_out"], B)
    a.update(kw)
    return a


def norm_args(**kw):
    x = torch.zeros(T, 512, dtype=BF16)
    a = dict(x=x, residual=torch.zeros(T, 512), gamma=torch.ones(512), out=torch.zeros(T, 512, dtype=BF16),
             out8=torch.zeros(T, 512, dtype=torch.uint8), out8_scale=torch.zeros(T, 4), sum=torch.zeros(T, 512))
    a["cfg"] = abi.make_add_rms_norm_config(x, a["residual"], a["out"], a["out8"], a["sum"], group=128)
    a.update(kw)
    return a


CALLS = [(abi.moe_add_rms_norm, norm_args), (abi.moe_blockkv_append, append_args), (abi.moe_blockkv_attention, attend_args),
         (abi.moe_blockkv_read, read_args)]


@pytest.mark.parametrize("call,args", CALLS)
def test_good_calls_pass_and_others_do_not(fake_lib, monkeypatch, call, args):   # noqa: F811
    call(**args())
    assert fake_lib.calls == 1
    for name, t in args().items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError, match="current CUDA device"):
                call(**args(**{name: elsewhere(t)}))
    monkeypatch.setattr(abi, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current CUDA device"):
        call(**args())
    assert fake_lib.calls == 1


@pytest.mark.parametrize("call,args", CALLS[1:])
def test_ragged_arrays_and_the_cache(fake_lib, call, args):   # noqa: F811
    for name in ("cu", "kv_len"):
        good = args()[name]
        for bad in (good.long(), good.float(), short(good)):
            with pytest.raises(ValueError, match=name):
                call(**args(**{name: bad}))
    with pytest.raises(ValueError, match="rows of the page table"):
        call(**args(cache=abi.make_blockkv_cache(**dict(cache_tensors(), page_table=torch.zeros(1, 4, dtype=I32)))))
    with pytest.raises(ValueError, match="current CUDA device"):
        call(**args(cache=abi.make_blockkv_cache(**{n: elsewhere(t) for n, t in cache_tensors().items()})))
    codes, scales = torch.zeros(9, HKV, PAGE, D, dtype=torch.uint8), torch.zeros(9, HKV, PAGE, D // 8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="cache's head"):
        call(**args(cache=abi.make_blockkv_cache(**dict(cache_tensors(), k=codes, v=codes, k_scale=scales, v_scale=scales))))
    assert fake_lib.calls == 0


def test_caches_that_are_none():
    t = cache_tensors()
    for name, bad in (("k", t["k"][:8]), ("v", t["v"].transpose(1, 2)), ("k_scale", t["k_scale"][..., :3]),
                      ("v_scale", t["v_scale"].float()), ("page_table", t["page_table"].long()),
                      ("page_table", torch.zeros(4, B, dtype=I32).T)):
        with pytest.raises(ValueError):
            abi.make_blockkv_cache(**dict(t, **{name: bad}))
    for dtype in (torch.float8_e4m3fn, torch.float8_e5m2):   # codes are bytes, scales E4M3 or bytes
        with pytest.raises(ValueError, match="two codes"):
            abi.make_blockkv_cache(**dict(t, k=t["k"].view(dtype), v=t["v"].view(dtype)))
    with pytest.raises(ValueError, match="E4M3"):
        abi.make_blockkv_cache(**dict(t, k_scale=t["k_scale"].view(torch.float8_e5m2), v_scale=t["v_scale"].view(torch.float8_e5m2)))
    for name in t:
        with pytest.raises(ValueError, match="one device"):
            abi.make_blockkv_cache(**{n: elsewhere(x) if n == name else x for n, x in t.items()})


def test_strides_of_a_cache():
    wide = torch.zeros(9, PAGE, HKV, 96, dtype=torch.uint8).transpose(1, 2)[..., :D // 2]
    scales = torch.zeros(9, PAGE, HKV, 8, dtype=torch.uint8).transpose(1, 2)[..., :D // 16]
    c = abi.make_blockkv_cache(wide, wide, scales, scales,
                               torch.zeros(B, 4, dtype=I32), k_gscale=0.25, v_gscale=4.0)
    assert (c.page_stride, c.head_stride, c.token_stride) == (PAGE * HKV * 96, 96, HKV * 96)
    assert (c.scale_page_stride, c.scale_head_stride, c.scale_token_stride) == (PAGE * HKV * 8, 8, HKV * 8)
    assert (c.k_gscale, c.v_gscale, c.head_dim, c.page_size, c.n_kv_heads, c.max_pages) == (0.25, 4.0, D, PAGE, HKV, 4)


@pytest.mark.parametrize("name,bad", [
    ("k", torch.zeros(T - 1, HKV, D, dtype=BF16)), ("gamma_k", torch.ones(D, dtype=BF16)), ("cos_sin", torch.zeros(49, D // 2, 2)),
    ("positions", torch.zeros(T, dtype=torch.int64)),
])
def test_append_types_and_sizes(fake_lib, name, bad):   # noqa: F811
    with pytest.raises(ValueError, match=name):
        abi.moe_blockkv_append(**append_args(**{name: bad}))
    assert fake_lib.calls == 0


@pytest.mark.parametrize("name,bad", [
    ("k_out", torch.zeros(T - 1, HKV, D, dtype=BF16)), ("v_out", torch.zeros(T, HKV, D)), ("k_out", torch.zeros(T, HKV, D, dtype=torch.float16)),
])
def test_read_types_and_sizes(fake_lib, name, bad):   # noqa: F811
    with pytest.raises(ValueError, match=name):
        abi.moe_blockkv_read(**read_args(**{name: bad}))
    assert fake_lib.calls == 0
    with pytest.raises(ValueError):
        abi.make_blockkv_read_config(None, None, 1)
    with pytest.raises(ValueError):
        abi.make_blockkv_read_config(torch.zeros(T, HKV, D), torch.zeros(T, HKV, D, dtype=BF16), 1)
    abi.moe_blockkv_read(**read_args(k_out=None))
    abi.moe_blockkv_read(**read_args(dtype=F32, v_out=None))
    assert fake_lib.calls == 2


@pytest.mark.parametrize("name,bad", [
    ("x", torch.zeros(T, 512)), ("x", torch.zeros(T - 1, 512, dtype=BF16)), ("x", torch.zeros(T, 1024, dtype=BF16)[:, :512]),
    ("residual", torch.zeros(T, 512, dtype=BF16)), ("sum", torch.zeros(T, 512, dtype=BF16)), ("out", torch.zeros(T, 504, dtype=BF16)),
    ("gamma", torch.ones(511)), ("gamma", torch.ones(512, dtype=BF16)), ("out8", torch.zeros(T, 504, dtype=torch.uint8)),
    ("out8_scale", torch.zeros(T, 3)), ("out8_scale", torch.zeros(T, 4, dtype=BF16)),
])
def test_norm_types_and_sizes(fake_lib, name, bad):   # noqa: F811
    with pytest.raises(ValueError, match=name):
        abi.moe_add_rms_norm(**norm_args(**{name: bad}))
    assert fake_lib.calls == 0


def test_norm_configurations(fake_lib):   # noqa: F811
    x = torch.zeros(T, 512, dtype=BF16)
    for kw in (dict(residual=x[:, :504]), dict(out=torch.zeros(T, 512, dtype=torch.float16)), dict(sum=x),
               dict(residual=x, sum=torch.zeros(T, 512)), dict(out8=torch.zeros(T, 512)), dict(out8=torch.zeros(T, 600, dtype=torch.uint8)[:, :512])):
        with pytest.raises(ValueError):
            abi.make_add_rms_norm_config(x, **kw)
    wide = torch.zeros(T, 1024, dtype=BF16)[:, 8:520]
    c = abi.make_add_rms_norm_config(wide, None, x)
    assert (c.x_stride, c.out_stride, c.d, c.T) == (1024, 512, 512, T)
    abi.moe_add_rms_norm(c, wide, None, torch.ones(512), x)
    with pytest.raises(ValueError):
        abi.moe_add_rms_norm(c, x, None, torch.ones(512), x)
    assert fake_lib.calls == 1
