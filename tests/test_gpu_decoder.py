"""The decoder layer over the paged cache: its operators together, prompt and
single tokens, against the fp64 oracles.

The layer's states pass bf16 about eight times (2^-9 each, two residual sums
carry them through), the attention weights f16, the cache E4M3 (compared with
the oracle's own cache, so its rounding is not an error): the output may be
off by about 1e-2 relative L2; 2e-2 is allowed.  The experts are compared on
the GPU's choice, which has to be a valid one."""
import numpy as np
import pytest
import torch

import moe_synth
import oracle
from oracle import decode_oracle as do
from top_routed_expert_gb300 import abi
from top_routed_expert_gb300.decoder import DecoderLayer, PagedKVCache
from top_routed_expert_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu

D, HQ, HKV, DM, E, K = 64, 8, 2, 256, 32, 4


def make(batch=3, page=16, window=0, n_sink=0, seed=0, scored=True):
    inp = moe_synth.make_custom(T=8, d=DM, E=E, k=K, f=128, fs=128, x_dtype="bf16", w_dtype="e4m3", seed=seed)
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    w_qkv = (rnd((HQ + 2 * HKV) * D, DM) / DM ** 0.5).to(torch.bfloat16)
    w_o = (rnd(DM, HQ * D) / (HQ * D) ** 0.5).to(torch.bfloat16)
    n1, n2, gq, gk = (torch.rand(n, generator=g) + 0.5 for n in (DM, DM, D, D))
    i = np.arange(D // 2)
    ang = np.arange(256)[:, None] * 10000.0 ** (-2.0 * i / D)
    cs = torch.from_numpy(np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32))
    moe = MoELayer(inp)
    route = dict(n_groups=4, top_groups=2, group_rank=2, score=abi.MOE_SCORE_SIGMOID, scale=1.5) if scored else {}
    cache = PagedKVCache(40, page, HKV, D, batch, 12)
    layer = DecoderLayer(moe, cache, w_qkv.cuda(), w_o.cuda(), n1.cuda(), n2.cuda(), cs.cuda(), HQ, gq.cuda(), gk.cuda(),
                         window=window, n_sink=n_sink, route=route)
    host = dict(inp=inp, w_qkv=w_qkv.double().numpy(), w_o=w_o.double().numpy(), n1=n1.double().numpy(),
                n2=n2.double().numpy(), gq=gq.double().numpy(), gk=gk.double().numpy(), cs=cs.double().numpy(),
                cache=do.Cache(np.zeros((40, HKV, page, D), dtype=np.uint8), np.zeros((40, HKV, page, D), dtype=np.uint8),
                               np.ones((40, HKV)), np.ones((40, HKV)), cache.table.cpu().numpy()), window=window,
                n_sink=n_sink)
    return layer, host


def bf(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def norm(x, gamma):
    return bf(x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6) * gamma)


def reference(layer, host, x, new, ids, w):
    """The layer in fp64 on the GPU's expert choice (ids, w), with the bf16 rounding of its states."""
    c = layer.cache
    host["cache"].table = c.table.cpu().numpy()
    cu = np.concatenate([[0], np.cumsum(new)])
    qkv = bf(norm(x, host["n1"]) @ host["w_qkv"].T)
    q, k, v = (y.reshape(len(x), -1, D) for y in np.split(qkv, [HQ * D, (HQ + HKV) * D], axis=1))
    q, _ = do.kv_append(host["cache"], q, k, v, host["gq"], host["gk"], host["cs"], None, cu, c.length)
    a, _ = do.paged_attention(host["cache"], bf(q), cu, c.length, D ** -0.5, host["window"], host["n_sink"])
    x = bf(x + bf(bf(a).reshape(len(x), -1) @ host["w_o"].T))
    h = norm(x, host["n2"])
    y = np.zeros_like(h)
    inp = host["inp"]
    weights = {}
    for t in range(len(h)):
        for e, g in zip(ids[t], w[t]):
            if e not in weights:
                weights[e] = oracle.expert_weights(inp, int(e))
            y[t] += g * oracle.swiglu_ffn(h[t:t + 1], *weights[e])[0]
    y += oracle.swiglu_ffn(h, *oracle.shared_weights(inp))
    return x + y, h


def run_steps(layer, host, steps, seed):
    g = torch.Generator().manual_seed(seed)
    for new in steps:
        x = torch.randn(sum(new), DM, generator=g).to(torch.bfloat16)
        chosen = []
        choose = layer.choose
        layer.choose = lambda h: chosen.append((h,) + choose(h)) or chosen[-1][1:]
        y = layer.forward(x.cuda(), list(new))
        layer.choose = choose
        assert abi.moe_get_device_status() == 0
        h, ids, w = (z.double().cpu().numpy() for z in chosen[0])
        ids = ids.astype(np.int64)
        ref, h_ref = reference(layer, host, x.double().numpy(), list(new), ids, w)
        got = y.double().cpu().numpy()
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= 2e-2, rel
        # a valid choice for the states that the GPU routed
        r = layer.route
        L = h @ host["inp"].w_router.astype(np.float64).T
        ref_ids, ref_w, choice = do.route_scores(L, host["inp"].bias, K, r.get("n_groups", 1), r.get("top_groups", 1),
                                                 r.get("group_rank", 1), "sigmoid" if r else "softmax", True,
                                                 r.get("scale", 1.0))
        same = np.mean(np.all(ids == ref_ids, axis=1))
        assert same >= 0.9 and np.all(np.abs(w.sum(1) - r.get("scale", 1.0)) <= 1e-5)


@pytest.mark.parametrize("scored", [True, False])
def test_prompt_then_tokens(scored):
    layer, host = make(scored=scored)
    run_steps(layer, host, [(37, 16, 5), (1, 1, 1), (1, 0, 1), (3, 1, 2), (40, 1, 1)], seed=1)


def test_sliding_window_with_sinks():
    layer, host = make(window=24, n_sink=2, seed=2)
    run_steps(layer, host, [(60, 3, 33), (1, 1, 1), (1, 1, 1)], seed=3)


def test_pages_come_back():
    layer, host = make(seed=4)
    c = layer.cache
    free = len(c.free)
    run_steps(layer, host, [(33, 16, 1)], seed=5)
    assert [len(p) for p in c.pages] == [3, 1, 1] and len(c.free) == free - 5
    c.release(0)
    assert len(c.free) == free - 2 and c.length[0] == 0
    run_steps(layer, host, [(20, 1, 1)], seed=6)
    with pytest.raises(ValueError):
        c.extend([200, 0, 0])
    with pytest.raises(ValueError):
        c.extend([1, 1])
