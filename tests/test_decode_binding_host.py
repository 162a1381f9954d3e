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
