"""Host-side checks of the decoder layer (no GPU needed): the library's calls
are replaced by the fp64 oracles, so what the layer passes to them shows."""
import inspect

import numpy as np
import pytest
import torch

import moe_synth
import oracle
from oracle import decode_oracle as do
from top_routed_expert_gb300 import abi
from top_routed_expert_gb300.decoder import DecoderLayer, PagedKVCache
from top_routed_expert_gb300.layer import MoELayer

D, HQ, HKV, DM, E, K = 64, 4, 2, 128, 32, 4


def make(skew=False, **kw):
    inp = moe_synth.make_custom(T=8, d=DM, E=E, k=K, f=64, fs=64, x_dtype="bf16", w_dtype="e4m3", seed=1, skew=skew)
    cache = PagedKVCache(12, 16, HKV, D, 2, 5, device="cpu")
    g = torch.Generator().manual_seed(2)
    w_qkv = (torch.randn((HQ + 2 * HKV) * D, DM, generator=g) / DM ** 0.5).to(torch.bfloat16)
    w_o = (torch.randn(DM, HQ * D, generator=g) / (HQ * D) ** 0.5).to(torch.bfloat16)
    one = torch.ones(DM)
    layer = DecoderLayer(MoELayer(inp, device="cpu"), cache, w_qkv, w_o, one, one, torch.zeros(80, D // 2, 2), HQ, **kw)
    return layer, inp


@pytest.fixture
def scores_by_oracle(monkeypatch):
    def call(cfg, logits, bias, ids, w, stream=None):
        a, b, _ = do.route_scores(logits.double().numpy(), None if bias is None else bias.numpy(), cfg.top_k, cfg.n_groups,
                                  cfg.top_groups, cfg.group_rank, "sigmoid" if cfg.score else "softmax",
                                  bool(cfg.renormalise), cfg.scale)
        ids.copy_(torch.from_numpy(a)), w.copy_(torch.from_numpy(b))
    monkeypatch.setattr(abi, "moe_route_scores", call)


def test_choice_of_a_biased_router_is_the_moe_layers(scores_by_oracle):
    """A MoELayer's bias belongs to its logits: it moves the choice and the gates."""
    layer, inp = make(skew=True)
    assert inp.bias is not None
    h = torch.randn(50, DM, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    ids, w = layer.choose(h)
    L, want, gates = oracle.route(h.double().numpy(), inp.w_router, inp.bias, K)
    clear = ~np.logical_or(*oracle.near_ties(L, K))   # fp32 logits are about 1e-6 off
    assert clear.sum() > 40 and np.array_equal(ids.numpy()[clear], want[clear])
    assert np.max(np.abs(w.double().numpy() - gates)[clear]) <= 1e-4


def test_choice_bias_moves_the_choice_alone(scores_by_oracle):
    b = torch.linspace(-0.3, 0.3, E)
    layer, inp = make(skew=True, choice_bias=b, route=dict(score=abi.MOE_SCORE_SIGMOID, n_groups=4, top_groups=2))
    h = torch.randn(50, DM, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    ids, w = layer.choose(h)
    L = h.double().numpy() @ inp.w_router.astype(np.float64).T + inp.bias
    want, gates, c = do.route_scores(L, b.numpy(), K, 4, 2, 1, "sigmoid")
    sorted_c = np.sort(c, axis=1)
    clear = np.min(np.diff(sorted_c, axis=1), axis=1) > 1e-5   # groups are ranked by the same values
    assert clear.sum() > 30 and np.array_equal(ids.numpy()[clear], want[clear])
    assert np.max(np.abs(w.double().numpy() - gates)[clear]) <= 1e-4


@pytest.mark.parametrize("stream", [None, "side"])
def test_routed_experts_allocate_on_the_stream_that_they_use(monkeypatch, stream):
    """What forward_routed drops at its end must belong to the stream whose kernels still use it."""
    current, seen = [None], []

    class use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            current.append(self.s)

        def __exit__(self, *_):
            current.pop()

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: seen.append(("alloc", current[-1])) or empty(*a, **kw))
    monkeypatch.setattr(abi, "moe_workspace_bytes", lambda cfg: 64)
    for name in ("moe_permute", "moe_expert_ffn", "moe_combine"):
        takes = len(inspect.signature(getattr(abi, name)).parameters)   # the last is the stream

        def call(*a, name=name, takes=takes, stream=None):
            seen.append((name, a[takes - 1] if len(a) == takes else stream or current[-1]))
        monkeypatch.setattr(abi, name, call)
    layer, _ = make()
    seen.clear()
    ids, w = torch.zeros(8, K, dtype=torch.int32), torch.zeros(8, K)
    layer.moe.forward_routed(torch.zeros(8, DM, dtype=torch.bfloat16), ids, w, stream=stream)
    assert {what for what, _ in seen} == {"alloc", "moe_permute", "moe_expert_ffn", "moe_combine"}
    assert {s for _, s in seen} == {stream}


def test_a_step_that_raises_can_be_made_again(monkeypatch):
    """The cache's lengths stay those of the tokens that were computed, whichever part of the step fails."""
    layer, _ = make()
    steps, fail = [], []

    def attention(h, cu, kv_len, max_q_len):
        steps.append((cu.tolist(), kv_len.tolist(), max_q_len))
        if fail == ["attention"]:
            raise abi.MoEError(4, "moe_paged_attention")
        return torch.zeros(h.shape[0], HQ, D, dtype=torch.bfloat16)

    def choose(h):
        if fail == ["choose"]:
            raise MemoryError
        return None, None
    monkeypatch.setattr(layer, "attention", attention)
    monkeypatch.setattr(layer, "choose", choose)
    monkeypatch.setattr(layer.moe, "forward_routed", lambda h, ids, w: torch.zeros(h.shape[0], DM))
    cache, x = layer.cache, torch.zeros(21, DM, dtype=torch.bfloat16)
    layer.forward(x[:18], [17, 1])
    assert cache.length == [17, 1]
    for what, error in (("attention", abi.MoEError), ("choose", MemoryError)):
        fail[:] = [what]
        with pytest.raises(error):
            layer.forward(x, [20, 1])
        assert cache.length == [17, 1]
        assert sorted(cache.free + cache.pages[0] + cache.pages[1]) == list(range(12))
    fail[:] = []
    layer.forward(x, [20, 1])
    assert cache.length == [37, 2] and steps[-1] == steps[1] == ([0, 20, 21], [37, 2], 20)
    assert [len(p) for p in cache.pages] == [3, 1]
    assert cache.table[0, :3].tolist() == cache.pages[0] and cache.table[0, 3:].eq(-1).all()


def test_room_that_cannot_be_made_changes_nothing():
    layer, _ = make()
    cache = layer.cache
    cache.extend([30, 5])
    before = cache.length[:], [p[:] for p in cache.pages], cache.free[:], cache.table.clone()
    for new, error in (([60, 0], ValueError), ([-1, 0], ValueError), ([1], ValueError)):
        with pytest.raises(error):
            cache.extend(new)
    cache.free, spare = [], cache.free
    with pytest.raises(RuntimeError):
        cache.extend([10, 0])
    cache.free = spare
    assert (cache.length, cache.pages, cache.free) == before[:3] and torch.equal(cache.table, before[3])
