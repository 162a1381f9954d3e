"""The decoder layer's expert choice on a biased router against the fused
router (moe_route) and the fp64 oracle: the same layer has to route alike
through MoELayer.forward and DecoderLayer.forward.

Both take fp32 logits, about 1e-6 off; a token whose oracle logits are within
1e-4 of each other at the edge of, or inside, its top k may differ.  Gates: a
softmax over the chosen logits, 1e-4 with that error."""
import numpy as np
import pytest
import torch

import moe_synth
import oracle
from top_routed_expert_gb300 import abi
from top_routed_expert_gb300.decoder import DecoderLayer, PagedKVCache
from top_routed_expert_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 256])
def test_choice_of_a_biased_router_is_that_of_moe_route(T):
    inp = moe_synth.make_custom(T=T, d=256, E=128, k=6, f=64, fs=64, x_dtype="bf16", w_dtype="e4m3", seed=5, skew=True)
    moe, one = MoELayer(inp), torch.ones(256, device="cuda")
    cache = PagedKVCache(4, 16, 1, 64, 1, 4)
    w = torch.zeros(3 * 64, 256, dtype=torch.bfloat16, device="cuda")
    layer = DecoderLayer(moe, cache, w, w[:64].T.contiguous(), one, one, torch.zeros(8, 32, 2, device="cuda"), 1)
    x = torch.from_numpy(inp.x.view(np.int16)).cuda().view(torch.bfloat16)
    ids, gates = (t.cpu().numpy() for t in layer.choose(x))
    fids = torch.empty(T, 6, dtype=torch.int32, device="cuda")
    fw = torch.empty(T, 6, device="cuda")
    abi.moe_route(moe.config(T), x, moe.w_router, moe.bias, fids, fw)
    assert abi.moe_get_device_status() == 0
    L, want, want_w = oracle.route(inp.x_f32, inp.w_router, inp.bias, 6)
    clear = ~np.logical_or(*oracle.near_ties(L, 6))
    assert clear.sum() >= 0.9 * T
    assert np.array_equal(ids[clear], want[clear]) and np.array_equal(fids.cpu().numpy()[clear], want[clear])
    assert np.max(np.abs(gates - want_w)[clear]) <= 1e-4
    assert np.max(np.abs(gates - fw.cpu().numpy())[clear]) <= 1e-4
