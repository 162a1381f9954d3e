"""Host-side checks of the decoder layer over the 4-bit cache (no GPU needed):
which operators it calls with what, and the cache's reads."""
import pytest
import torch

import moe_synth
from tests.test_decoder_host import D, DM, E, HKV, HQ, K
from top_routed_expert_gb300 import abi
from top_routed_expert_gb300.decoder import DecoderLayer, PagedBlockKVCache, PagedKVCache, rms_norm
from top_routed_expert_gb300.layer import MoELayer


def make(kind, **kw):
    inp = moe_synth.make_custom(T=8, d=DM, E=E, k=K, f=64, fs=64, x_dtype="bf16", w_dtype="e4m3", seed=1)
    cache = kind(12, 16, HKV, D, 2, 5, device="cpu")
    g = torch.Generator().manual_seed(2)
    w_qkv = (torch.randn((HQ + 2 * HKV) * D, DM, generator=g) / DM ** 0.5).to(torch.bfloat16)
    w_o = (torch.randn(DM, HQ * D, generator=g) / (HQ * D) ** 0.5).to(torch.bfloat16)
    gamma = torch.rand(DM, generator=g) + 0.5
    return DecoderLayer(MoELayer(inp, device="cpu"), cache, w_qkv, w_o, gamma, gamma, torch.zeros(80, D // 2, 2), HQ, **kw)


@pytest.mark.parametrize("kind,prefix", [(PagedKVCache, ""), (PagedBlockKVCache, "block")])
def test_each_cache_has_its_own_operators(monkeypatch, kind, prefix):
    layer, seen = make(kind), []
    names = {"": ("moe_kv_append", "moe_paged_attention", "moe_paged_attention_ws_bytes"),
             "block": ("moe_blockkv_append", "moe_blockkv_attention", "moe_blockkv_attention_ws_bytes")}
    for kinds in names.values():
        for name in kinds:
            monkeypatch.setattr(abi, name, lambda cfg, cache, *a, name=name: seen.append((name, cache, len(a))) or 64)
    h = torch.zeros(5, DM, dtype=torch.bfloat16)
    cu, kv_len = layer.cache.extend([4, 1])
    out = layer.attention(h, cu, kv_len, 4)
    assert out.shape == (5, HQ, D)
    append, attend, size = names[prefix]
    assert [s[0] for s in seen] == [append, size, attend]
    assert all(s[1] is layer.cache.handle for s in seen) and seen[0][2] == 10 and seen[2][2] == 6


def test_norms_of_the_library(monkeypatch):
    """With fused_norm both norms and the first addition go to moe_add_rms_norm, and the values are the same."""
    plain, fused = make(PagedBlockKVCache), make(PagedBlockKVCache, fused_norm=True)
    calls = []

    def call(cfg, x, residual, gamma, out=None, out8=None, out8_scale=None, sum=None, stream=None):
        calls.append(cfg)
        h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
        if sum is not None:
            sum.copy_(h)
        out.copy_(rms_norm(h, gamma, cfg.eps))
    monkeypatch.setattr(abi, "moe_add_rms_norm", call)
    for layer in (plain, fused):
        monkeypatch.setattr(layer, "attention", lambda h, cu, kv_len, n: h[:, :HQ * D // 4].reshape(-1, HQ, D // 4).repeat(1, 1, 4))
        monkeypatch.setattr(layer, "choose", lambda h: (None, None))
        monkeypatch.setattr(layer.moe, "forward_routed", lambda h, ids, w: h.float() * 0.5)
    x = torch.randn(6, DM, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    assert torch.equal(plain.forward(x, [5, 1]), fused.forward(x, [5, 1]))
    assert len(calls) == 2 and all(c.T == 6 and c.d == DM and c.out_dtype == abi.MOE_BF16 for c in calls)


def test_reads(monkeypatch):
    cache, seen = PagedBlockKVCache(12, 16, HKV, D, 2, 5, device="cpu", k_gscale=0.5, v_gscale=2.0), []
    assert (cache.handle.k_gscale, cache.handle.v_gscale) == (0.5, 2.0)
    cache.extend([20, 3])
    monkeypatch.setattr(abi, "moe_blockkv_read", lambda cfg, c, cu, ln, k, v: seen.append((cu.tolist(), ln.tolist(), k, v, cfg, c)))
    cu, k, v = cache.read()
    assert cu == [0, 20, 23] and k.shape == v.shape == (23, HKV, D) and k.dtype == torch.bfloat16
    assert seen[0][:2] == ([0, 20, 23], [20, 3]) and seen[0][5] is cache.handle
    cu, k, v = cache.read([0, 2], torch.float32)
    assert cu == [0, 0, 2] and k.dtype == torch.float32 and seen[1][:2] == ([0, 0, 2], [20, 3])
    for bad in ([21, 0], [0, -1], [1]):
        with pytest.raises(ValueError):
            cache.read(bad)


def test_memory():
    """9/16 of the 8-bit cache's codes, and as large whatever the factors are."""
    a, b = PagedKVCache(12, 16, HKV, 128, 2, 5, device="cpu"), PagedBlockKVCache(12, 16, HKV, 128, 2, 5, device="cpu")
    assert 16 * (b.k.nbytes + b.k_scale.nbytes) == 9 * a.k.nbytes
    with pytest.raises(ValueError):
        abi.make_blockkv_cache(b.k, b.v, a.k_scale, a.v_scale, b.table)
