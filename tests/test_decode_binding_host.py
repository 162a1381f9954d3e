"""Host-side checks of the binding of the decoder-step operators (abi.py): what
the kernels assume of the tensors that a call names is refused before the
library is called.  No GPU: the tensors are on the CPU, a stand-in says that
this is the current device, and another stand-in takes the calls."""
import pytest
import torch

from top_routed_expert_gb300 import abi

I32, BF16, F32 = torch.int32, torch.bfloat16, torch.float32
T, B, HQ, HKV, D, PAGE = 5, 2, 6, 2, 64, 16


class Library:
    """Takes every call and counts them."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*a):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(abi, "load", lambda: fake)
    monkeypatch.setattr(abi, "_current_device", lambda: -1)      # of a CPU tensor
    monkeypatch.setattr(abi, "_current_stream", lambda dev: 0)
    return fake


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another device."""

    def get_device(self):
        return 1


def elsewhere(t):
    return t.as_subclass(Elsewhere)


def route_args(**kw):
    a = dict(cfg=abi.make_route_scores_config(T, 128, 6), logits=torch.zeros(T, 128), bias=torch.zeros(128),
             topk_ids=torch.zeros(T, 6, dtype=I32), topk_w=torch.zeros(T, 6))
    a.update(kw)
    return a


def cache_tensors():
    codes = torch.zeros(9, HKV, PAGE, D, dtype=torch.uint8)
    return dict(k=codes, v=codes.clone(), k_scale=torch.ones(9, HKV), v_scale=torch.ones(9, HKV),
                page_table=torch.zeros(B, 4, dtype=I32))


def append_args(**kw):
    q, k = torch.zeros(T, HQ, D, dtype=BF16), torch.zeros(T, HKV, D, dtype=BF16)
    a = dict(q=q, k=k, v=k.clone(), gamma_q=torch.ones(D), gamma_k=torch.ones(D), cos_sin=torch.zeros(50, D // 2, 2),
             positions=torch.zeros(T, dtype=I32), cu=torch.zeros(B + 1, dtype=I32), kv_len=torch.zeros(B, dtype=I32),
             q_out=torch.zeros_like(q), cache=abi.make_kv_cache(**cache_tensors()))
    a["cfg"] = abi.make_kv_append_config(a["q"], a["k"], a["v"], a["q_out"], B, rot_dim=D, n_pos=50)
    a.update(kw)
    return a


def attend_args(**kw):
    q = torch.zeros(T, HQ, D, dtype=BF16)
    a = dict(q=q, cu=torch.zeros(B + 1, dtype=I32), kv_len=torch.zeros(B, dtype=I32), out=torch.zeros_like(q),
             lse=torch.zeros(T, HQ), ws=torch.zeros(64, dtype=torch.uint8), cache=abi.make_kv_cache(**cache_tensors()))
    a["cfg"] = abi.make_paged_attention_config(a["q"], a["out"], B)
    a.update(kw)
    return a


CALLS = [(abi.moe_route_scores, route_args), (abi.moe_kv_append, append_args), (abi.moe_paged_attention, attend_args)]


@pytest.mark.parametrize("call,args", CALLS)
def test_good_calls_pass(lib, call, args):
    call(**args())
    assert lib.calls == 1


# ----------------------------------------------------------------- devices

@pytest.mark.parametrize("call,args", CALLS)
def test_tensors_of_another_device(lib, monkeypatch, call, args):
    for name, t in args().items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError, match="current CUDA device"):
                call(**args(**{name: elsewhere(t)}))
    monkeypatch.setattr(abi, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current CUDA device"):
        call(**args())
    assert lib.calls == 0


@pytest.mark.parametrize("call,args", CALLS[1:])
def test_cache_of_another_device(lib, call, args):
    with pytest.raises(ValueError, match="current CUDA device"):
        call(**args(cache=abi.make_kv_cache(**{n: elsewhere(t) for n, t in cache_tensors().items()})))
    for name in cache_tensors():
        with pytest.raises(ValueError, match="one device"):
            abi.make_kv_cache(**{n: elsewhere(t) if n == name else t for n, t in cache_tensors().items()})
    assert lib.calls == 0


def test_stream_of_another_device():
    class Stream:
        device_index, cuda_stream = 1, 77
    assert abi._stream_of(Stream(), 1) == 77
    with pytest.raises(ValueError, match="current CUDA device"):
        abi._stream_of(Stream(), 0)


# ----------------------------------------------------------------- types and lengths

def short(t):
    return t.flatten()[:-1]


@pytest.mark.parametrize("call,args", CALLS[1:])
def test_offsets_and_lengths(lib, call, args):
    for name in ("cu", "kv_len"):
        good = args()[name]
        for bad in (good.long(), good.float(), short(good)):
            with pytest.raises(ValueError, match=name):
                call(**args(**{name: bad}))
    assert lib.calls == 0


@pytest.mark.parametrize("call,args", CALLS[1:])
def test_more_requests_than_the_page_table_has(lib, call, args):
    one = cache_tensors()
    one["page_table"] = one["page_table"][:1]
    with pytest.raises(ValueError, match="rows of the page table"):
        call(**args(cache=abi.make_kv_cache(**one)))
    cfg = args()["cfg"]
    cfg.batch = B + 1
    with pytest.raises(ValueError, match="rows of the page table"):
        call(**args(cfg=cfg, cu=torch.zeros(9, dtype=I32), kv_len=torch.zeros(9, dtype=I32)))
    assert lib.calls == 0


@pytest.mark.parametrize("name,bad", [
    ("logits", torch.zeros(T, 128, dtype=BF16)), ("logits", torch.zeros(T, 128, dtype=torch.float64)),
    ("logits", torch.zeros(T - 1, 128)), ("bias", torch.zeros(127)), ("bias", torch.zeros(128, dtype=BF16)),
    ("topk_ids", torch.zeros(T, 6, dtype=torch.int64)), ("topk_ids", torch.zeros(T, 5, dtype=I32)),
    ("topk_w", torch.zeros(T, 6, dtype=BF16)), ("topk_w", torch.zeros(T - 1, 6)),
])
def test_route_scores_types_and_sizes(lib, name, bad):
    with pytest.raises(ValueError, match=name):
        abi.moe_route_scores(**route_args(**{name: bad}))
    assert lib.calls == 0


def test_route_scores_logits_of_the_configured_type(lib):
    cfg = abi.make_route_scores_config(T, 128, 6, logit_dtype=abi.MOE_BF16)
    abi.moe_route_scores(**route_args(cfg=cfg, logits=torch.zeros(T, 128, dtype=BF16), bias=None))
    assert lib.calls == 1
    with pytest.raises(ValueError, match="logits"):
        abi.moe_route_scores(**route_args(cfg=cfg))
    assert lib.calls == 1


def test_route_scores_rows_apart(lib):
    cfg = abi.make_route_scores_config(T, 128, 6, logit_stride=140)
    abi.moe_route_scores(**route_args(cfg=cfg, logits=torch.zeros(T, 140)[:, :128]))
    abi.moe_route_scores(**route_args(cfg=cfg, logits=torch.zeros(T, 140)))
    assert lib.calls == 2
    for bad in (torch.zeros(T, 128), torch.zeros(T, 139)[:, :128], torch.zeros(T - 1, 140)[:, :128]):
        with pytest.raises(ValueError, match="logits"):
            abi.moe_route_scores(**route_args(cfg=cfg, logits=bad))
    assert lib.calls == 2


def test_a_configuration_of_fewer_rows(lib):
    """The fields are the caller's: fewer rows than it was made from take shorter tensors."""
    a, c = append_args(), attend_args()
    a["cfg"].T = c["cfg"].T = T - 2
    abi.moe_kv_append(**dict(a, **{n: a[n][:T - 2] for n in ("q", "k", "v", "q_out", "positions")}))
    abi.moe_paged_attention(**dict(c, **{n: c[n][:T - 2] for n in ("q", "out", "lse")}))
    assert lib.calls == 2


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(T - 1, HQ, D, dtype=BF16)), ("q_out", torch.zeros(T, HQ - 1, D, dtype=BF16)),
    ("k", torch.zeros(T - 1, HKV, D, dtype=BF16)), ("v", torch.zeros(T, 1, D, dtype=BF16)),
    ("gamma_q", torch.ones(D - 1)), ("gamma_k", torch.ones(D, dtype=BF16)), ("gamma_k", torch.ones(D // 2)),
    ("cos_sin", torch.zeros(49, D // 2, 2)), ("cos_sin", torch.zeros(50, D // 2, 2, dtype=BF16)),
    ("positions", torch.zeros(T - 1, dtype=I32)), ("positions", torch.zeros(T, dtype=torch.int64)),
])
def test_kv_append_types_and_sizes(lib, name, bad):
    with pytest.raises(ValueError, match=name):
        abi.moe_kv_append(**append_args(**{name: bad}))
    assert lib.calls == 0


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(T - 1, HQ, D, dtype=BF16)), ("out", torch.zeros(T, HQ - 1, D, dtype=BF16)),
    ("lse", torch.zeros(T, HQ - 1)), ("lse", torch.zeros(T, HQ, dtype=BF16)),
])
def test_paged_attention_types_and_sizes(lib, name, bad):
    with pytest.raises(ValueError, match=name):
        abi.moe_paged_attention(**attend_args(**{name: bad}))
    assert lib.calls == 0


def test_heads_of_another_cache(lib):
    other = torch.zeros(9, HKV, PAGE, 2 * D, dtype=torch.uint8)
    c = abi.make_kv_cache(**dict(cache_tensors(), k=other, v=other))
    for call, args in CALLS[1:]:
        with pytest.raises(ValueError, match="cache's head"):
            call(**args(cache=c))
    assert lib.calls == 0


def test_what_may_be_left_out(lib):
    abi.moe_route_scores(**route_args(bias=None))
    k = torch.zeros(T, HKV, D, dtype=BF16)
    abi.moe_kv_append(**append_args(cfg=abi.make_kv_append_config(None, k, k, None, B), q=None, q_out=None, gamma_q=None,
                                    gamma_k=None, cos_sin=None, positions=None))
    abi.moe_paged_attention(**attend_args(lse=None, ws=None))
    # arrays of a longer call serve shorter ones
    abi.moe_paged_attention(**attend_args(cu=torch.zeros(99, dtype=I32), kv_len=torch.zeros(99, dtype=I32),
                                          lse=torch.zeros(2 * T, HQ)))
    assert lib.calls == 4


def test_caches_of_other_8_bit_types():
    for dtype in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.bool):
        codes = torch.zeros(9, HKV, PAGE, D, dtype=torch.uint8).view(dtype)
        with pytest.raises(ValueError, match="E4M3"):
            abi.make_kv_cache(**dict(cache_tensors(), k=codes, v=codes))


def test_queries_and_keys_of_two_head_sizes():
    q, k = torch.zeros(T, HQ, 2 * D, dtype=BF16), torch.zeros(T, HKV, D, dtype=BF16)
    with pytest.raises(ValueError, match="head size"):
        abi.make_kv_append_config(q, k, k, q, B)
