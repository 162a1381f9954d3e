"""The decoder layer over the 4-bit cache, its operators together: prompts and
single tokens, against the fp64 oracles.

As in the test over the 8-bit cache the states pass bf16 about eight times: 1e-2
relative L2 is expected, 2e-2 allowed.  Keys and values are those that the GPU's
cache holds (a key next to a code's border may be either code when the states
before it differ by a rounding); what it holds is checked against the fp64 keys
and values: half of E2M1's widest step, 1 of 6, of a scale that is at most 9/8 of
the block's largest element / 6, so 3/16 of that element, and 2^-6 of the row's
largest for the bf16 states before."""
import numpy as np
import pytest
import torch

import oracle
from oracle import decode_oracle as do
from tests.test_gpu_decoder import D, DM, HKV, HQ, K, bf, make, norm
from top_routed_expert_gb300 import abi
from top_routed_expert_gb300.decoder import DecoderLayer, PagedBlockKVCache

pytestmark = pytest.mark.gpu


def over_blocks(page, fused, window=0, n_sink=0, seed=0):
    layer, host = make(page=page, window=window, n_sink=n_sink, seed=seed)
    cache = PagedBlockKVCache(40, page, HKV, D, 3, 12, k_gscale=0.5, v_gscale=0.125)
    return DecoderLayer(layer.moe, cache, layer.w_qkv, layer.w_o, layer.norm_attn, layer.norm_moe, layer.cos_sin, HQ,
                        layer.gamma_q, layer.gamma_k, window=window, n_sink=n_sink, route=layer.route, fused_norm=fused), host


class Held:
    """What the GPU's cache holds, as the attention oracle reads it."""

    def __init__(self, cache):
        cu, k, v = cache.read(dtype=torch.float32)
        self.rows = {"k": k.double().cpu().numpy(), "v": v.double().cpu().numpy()}
        self.cu, self.codes = cu, {"k": np.zeros((1, HKV, 1, D))}

    def values(self, which, b, h, n):
        return self.rows[which][self.cu[b]:self.cu[b] + n, h]


def step(layer, host, exact, new, g):
    x = torch.randn(sum(new), DM, generator=g).to(torch.bfloat16)
    chosen, choose = [], layer.choose
    layer.choose = lambda h: chosen.append(choose(h)) or chosen[-1]
    y = layer.forward(x.cuda(), list(new))
    layer.choose = choose
    assert abi.moe_get_device_status() == 0
    ids, w = (z.double().cpu().numpy() for z in chosen[0])
    x = x.double().numpy()
    cu = np.concatenate([[0], np.cumsum(new)])
    qkv = bf(norm(x, host["n1"]) @ host["w_qkv"].T)
    q, k, v = (z.reshape(len(x), -1, D) for z in np.split(qkv, [HQ * D, (HQ + HKV) * D], axis=1))
    c, held = layer.cache, Held(layer.cache)
    for b, n in enumerate(new):
        for i in range(n):
            t, pos = cu[b] + i, c.length[b] - n + i
            q[t] = do.norm_rotate(q[t], host["gq"], host["cs"][pos], "half", 1e-6)
            exact["k"][b].append(do.norm_rotate(k[t], host["gk"], host["cs"][pos], "half", 1e-6))
            exact["v"][b].append(v[t].copy())
    for name in "kv":
        for b in range(3):
            want, got = np.array(exact[name][b]).reshape(-1, HKV, D), held.rows[name][held.cu[b]:held.cu[b + 1]]
            top = np.repeat(np.max(np.abs(want.reshape(-1, HKV, D // 16, 16)), -1), 16, -1)
            bound = 3 / 16 * top + 2.0 ** -6 * np.max(np.abs(want), -1, keepdims=True) if len(want) else 0
            assert want.shape == got.shape and np.all(np.abs(got - want) <= bound)
    a, _ = do.paged_attention(held, bf(q), cu, c.length, D ** -0.5, host["window"], host["n_sink"])
    x = bf(x + bf(bf(a).reshape(len(x), -1) @ host["w_o"].T))
    h = norm(x, host["n2"])
    out, inp, weights = oracle.swiglu_ffn(h, *oracle.shared_weights(host["inp"])), host["inp"], {}
    for t in range(len(h)):
        for e, gate in zip(ids[t].astype(int), w[t]):
            if e not in weights:
                weights[e] = oracle.expert_weights(inp, int(e))
            out[t] += gate * oracle.swiglu_ffn(h[t:t + 1], *weights[e])[0]
    got, ref = y.double().cpu().numpy(), x + out
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= 2e-2, rel
    assert ids.shape == (len(x), K)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("page,window,n_sink", [(16, 0, 0), (32, 24, 2)])
def test_prompts_then_tokens(page, window, n_sink, fused):
    layer, host = over_blocks(page, fused, window, n_sink, seed=page)
    exact, g = {"k": [[], [], []], "v": [[], [], []]}, torch.Generator().manual_seed(1)
    for new in [(37, 16, 5), (1, 1, 1), (1, 0, 1), (3, 1, 2), (40, 1, 1)]:
        step(layer, host, exact, new, g)


def test_fused_norms_change_roundings_alone():
    """The same steps with and without: the states between differ by bf16 roundings, the outputs by 2e-2 at most."""
    outs = []
    for fused in (False, True):
        layer, _ = over_blocks(16, fused, seed=3)
        g = torch.Generator().manual_seed(4)
        for new in [(33, 16, 1), (1, 1, 1)]:
            outs.append(layer.forward(torch.randn(sum(new), DM, generator=g).to(torch.bfloat16).cuda(), list(new)).double())
    for a, b in zip(outs[:2], outs[2:]):
        assert (a - b).norm() <= 2e-2 * a.norm()
    free = len(layer.cache.free)
    layer.cache.release(0)
    assert len(layer.cache.free) == free + 3
