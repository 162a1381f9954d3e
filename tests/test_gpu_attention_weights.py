"""GPU parity of moe_paged_attention (include/paged_kv.h) on long contexts in
which a few tokens take almost all of the softmax but have no value, so that
the output is what the many small weights leave.  Compared relative to the row's
own exact output.

All values are positive, so relative errors of the weights carry over to the
output: f16 (2^-11) and fp32 scores (about 1e-5), then one bf16 rounding (2^-9),
together under 2^-8 |ref|.  Weights under 2^-22 of the row's largest lose up to
2^-33 of it: tokens 2^-33 max_j(softmax_j scale_j) max|code| more.
lse as in the other attention tests."""
import math

import pytest
import torch

from top_routed_expert_gb300 import abi

pytestmark = pytest.mark.gpu

J, PAGE, GROUP = 65536, 64, 8


def shared_context(D, nats, octaves, seed):
    """One context of J tokens, for every request the same.  Tokens 0, 16, 32 and 48 (nats > 0) score about `nats` above
    the others and have zero values; the value scale of their page is 2^octaves times that of the others."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    n = J // PAGE
    k = (rnd(n, 1, PAGE, D) * 30).clamp(-448, 448)
    v = 1 + 0.25 * rnd(n, 1, PAGE, D)
    vs = torch.full((n, 1), 2.0 ** -6, device="cuda")
    vs[0] *= 2.0 ** octaves
    v = v.clamp(min=0.25) / vs[:, :, None, None]
    if nats:
        k[0, 0, ::16] = nats / D ** 0.5 * 64
        v[0, 0, ::16] = 0
    k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    order = torch.randperm(n, generator=g, device="cuda")   # where page i lies
    at = torch.argsort(order)
    ks = torch.full((n, 1), 2.0 ** -6, device="cuda")
    move = lambda x: x.view(torch.uint8)[at].contiguous().view(torch.float8_e4m3fn)
    return move(k), move(v), ks, vs[at].contiguous(), order.to(torch.int32)


def run(D, new, batch, nats, octaves, seed=0):
    k, v, ks, vs, order = shared_context(D, nats, octaves, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    q1 = (1 + 0.25 * torch.randn(new, GROUP, D, generator=g, device="cuda")).to(torch.bfloat16)
    q = q1.repeat(batch, 1, 1)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * new
    kv_len = torch.full((batch,), J, dtype=torch.int32, device="cuda")
    table = order[None].repeat(batch, 1).contiguous()
    cache = abi.make_kv_cache(k, v, ks, vs, table)
    cfg = abi.make_paged_attention_config(q, out, batch, max_q_len=new)
    ws = torch.empty(abi.moe_paged_attention_ws_bytes(cfg, cache), dtype=torch.uint8, device="cuda")
    abi.moe_paged_attention(cfg, cache, q, cu, kv_len, out, lse, ws)
    assert abi.moe_get_device_status() == 0
    # the first request in 64 bits, some rows at a time
    where = order.long()
    K = (k[where].double() * ks[where].double()[..., None, None]).reshape(J, D)
    codes, scale = v[where].double().reshape(J, D), vs[where].double().repeat_interleave(PAGE, 0)[:, 0]
    V = codes * scale[:, None]
    j = torch.arange(J, device="cuda")
    ref, ref_l, lost = [], [], []
    for t in range(0, new, 16):
        z = (q1[t:t + 16].double() @ K.T) * D ** -0.5
        pos = J - new + torch.arange(t, min(new, t + 16), device="cuda")
        z.masked_fill_((j > pos[:, None])[:, None], -math.inf)
        p = torch.softmax(z, -1)
        ref.append(p @ V), ref_l.append(torch.logsumexp(z, -1)), lost.append((p * scale).amax(-1))
    ref, ref_l, lost = torch.cat(ref), torch.cat(ref_l), torch.cat(lost)
    bound = 2.0 ** -8 * ref.abs() + (J * 2.0 ** -33 * codes.abs().max() * lost)[..., None]
    assert torch.all(ref > 0)
    if nats:
        assert torch.all(bound < 0.2 * ref)   # nothing of the size of the output may be missing
    got = out.double().view(batch, new, GROUP, D)
    assert torch.all((got - ref).abs() <= bound), ((got - ref).abs() / ref).max()
    assert torch.all((lse.double().view(batch, new, GROUP) - ref_l).abs() <= 2e-5 * (1 + ref_l.abs().max()))


WEIGHTS = [(0.0, 0), (18.0, 0), (12.5, 8)]   # nothing stands out; weights of e^-18; of e^-12.5 at 2^-8 of the scale


@pytest.mark.parametrize("nats,octaves", WEIGHTS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_tokens(D, nats, octaves):
    # as many requests as CTAs, so that most warps go through a whole context
    run(D, 1, 608, nats, octaves)


@pytest.mark.parametrize("nats,octaves", WEIGHTS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompts(D, nats, octaves):
    # so many row blocks that none is cut along the tokens
    run(D, 128, 164, nats, octaves)
