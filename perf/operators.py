"""Cases, plain forms and 64-bit forms of the operators around the MoE layer in a decoder step.

  route   expert selection from router logits: softmax or sigmoid scores, a balance bias, expert groups, top-k,
          renormalised weights
  append  new keys and values into a paged cache of E4M3 codes with one scale per page and head; the QK norm and the
          rotation are applied on the way, to the queries as well
  attend  attention of the new queries over that cache: causal, grouped heads, optional sliding window with a few
          first tokens that stay visible

`own` chooses between the plain torch form and the library's calls."""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of the 128-expert top-6 layer: the latency of a single decode stream
        dict(name="route 1x128 softmax", op="route", T=1, E=128, k=6, G=1, tg=1, rank=1, score="softmax", bias=False,
             scale=1.0, dtype="f32", norm=True),
        # a decode batch with grouped sigmoid routing and a balance bias
        dict(name="route 64x256 groups", op="route", T=64, E=256, k=8, G=8, tg=4, rank=2, score="sigmoid", bias=True,
             scale=2.5, dtype="f32", norm=True),
        # a long prefill step of the same router, logits in bf16, an odd number of tokens
        dict(name="route 65519x256 groups", op="route", T=65519, E=256, k=8, G=8, tg=4, rank=2, score="sigmoid",
             bias=True, scale=2.5, dtype="bf16", norm=True),
        # a decode step: one new token for each of 64 requests, 32 query and 4 key heads of 128
        dict(name="append decode 64", op="append", batch=64, q_len=1, ragged=False, ctx_min=17, ctx_max=3712, Hq=32,
             Hkv=4, D=128, rot=128, layout="half", norm=True, page=16),
        # chunked prefill: 32 requests, 256 tokens each
        dict(name="append prefill 32x256", op="append", batch=32, q_len=256, ragged=False, ctx_min=256, ctx_max=3584,
             Hq=32, Hkv=4, D=128, rot=128, layout="half", norm=True, page=16),
        # ragged prompts, interleaved pairs on half of a 64-wide head, every head its own keys, larger pages
        dict(name="append ragged interleaved", op="append", batch=23, q_len=1999, ragged=True, ctx_min=2000,
             ctx_max=4003, Hq=16, Hkv=16, D=64, rot=32, layout="interleaved", norm=False, page=64),
        # one request, one token, a 3584-token prompt behind it
        dict(name="attend decode 1x3585", op="attend", batch=1, q_len=1, ragged=False, ctx_min=3585, ctx_max=3585,
             Hq=32, Hkv=4, D=128, window=0, sinks=0, page=16),
        # a decode batch of 64 requests at mixed lengths
        dict(name="attend decode 64x3712", op="attend", batch=64, q_len=1, ragged=False, ctx_min=17, ctx_max=3712,
             Hq=32, Hkv=4, D=128, window=0, sinks=0, page=16),
        # long contexts: 12 requests of up to 65536 tokens
        dict(name="attend decode 12x65536", op="attend", batch=12, q_len=1, ragged=False, ctx_min=49157,
             ctx_max=65536, Hq=32, Hkv=4, D=128, window=0, sinks=0, page=64),
        # a sliding window with 4 sinks, up to 4 tokens a request (a draft being checked), heads of 64
        dict(name="attend window draft", op="attend", batch=48, q_len=4, ragged=True, ctx_min=5, ctx_max=16381, Hq=32,
             Hkv=8, D=64, window=1024, sinks=4, page=32),
        # chunked prefill: 32 requests, 256 tokens each, over what they have so far
        dict(name="attend prefill 32x256", op="attend", batch=32, q_len=256, ragged=False, ctx_min=256, ctx_max=3584,
             Hq=32, Hkv=4, D=128, window=0, sinks=0, page=16),
        # ragged prompts in one batch, some long and some of a few tokens
        dict(name="attend prefill ragged", op="attend", batch=7, q_len=2047, ragged=True, ctx_min=2047, ctx_max=4093,
             Hq=16, Hkv=4, D=128, window=0, sinks=0, page=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "append", "attend", "attend"])
    if op == "route":
        E, G = rng.choice([(8, 1), (60, 1), (64, 8), (72, 3), (128, 1), (128, 8), (160, 8), (256, 1), (256, 8)])
        tg = rng.randint(1, G)
        k = rng.randint(1, min(16, tg * (E // G)))
        return dict(op=op, T=_log_int(rng, 1, 65519), E=E, k=k, G=G, tg=tg, rank=rng.choice([1, 2]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.8)
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8, 16])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    Hq = Hkv * group
    if op == "append":
        q_len = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2000)
        batch = _log_int(rng, 1, min(256, max(1, 2 ** 25 // (q_len * (Hq + 2 * Hkv) * D))))
        ctx_max = q_len + _log_int(rng, 1, 2048)
        return dict(op=op, batch=batch, q_len=q_len, ragged=rng.random() < 0.5, ctx_min=rng.randint(q_len, ctx_max),
                    ctx_max=ctx_max, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2]),
                    layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5, page=page)
    if rng.random() < 0.6:
        q_len = rng.choice([1, 1, 1, 2, 4, 7])
        ctx_max = q_len + _log_int(rng, 1, 65530)
        batch = _log_int(rng, 1, min(256, max(1, 2 ** 28 // (ctx_max * Hkv * D))))
    else:
        q_len = min(_log_int(rng, 16, 2047), 2 ** 16 // Hq)
        ctx_max = q_len + _log_int(rng, 1, 4096)
        batch = _log_int(rng, 1, max(1, 2 ** 28 // (q_len * Hq * ctx_max)))
    window = 0 if rng.random() < 0.6 else _log_int(rng, 1, 4096)
    return dict(op=op, batch=batch, q_len=q_len, ragged=rng.random() < 0.5, ctx_min=rng.randint(q_len, ctx_max),
                ctx_max=ctx_max, Hq=Hq, Hkv=Hkv, D=D, window=window,
                sinks=rng.choice([0, 1, 4, 16]) if window else 0, page=page)


def _lengths(c):
    """(new tokens, tokens in the cache with them) of each request: spread over the case's range, the order mixed."""
    B = c["batch"]
    mix = [(b * 7919 + 3) % B for b in range(B)]
    n = [1 + (c["q_len"] - 1) * (B - 1 - m) // max(1, B - 1) if c["ragged"] else c["q_len"] for m in mix]
    total = [c["ctx_max"] - (c["ctx_max"] - c["ctx_min"]) * ((m * 31 + 7) % B) // max(1, B - 1) for m in mix]
    return n, total


def _seen(n, total, window, sinks):
    """Tokens that the last query and, summed, all n queries of a request see; cached tokens that any of them sees."""
    pairs = 0
    for i in range(n):
        p = total - n + i
        pairs += p + 1 if not window or window > p else window + min(sinks, p + 1 - window)
    first = total - n
    union = total if not window or window > first else total - (first - window + 1) + min(sinks, first - window + 1)
    return pairs, union


def work(c):
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * (4 if c["dtype"] == "f32" else 2) + E * 4 * c["bias"] + T * k * 8,
                "flops": T * E * 6}
    n, total = _lengths(c)
    T, D, Hq, Hkv = sum(n), c["D"], c["Hq"], c["Hkv"]
    if c["op"] == "append":
        blocks = sum((t - 1) // c["page"] - (t - m) // c["page"] + 1 for m, t in zip(n, total))
        return {"bytes": T * (2 * Hq * D * 2 + Hkv * D * (4 + 2)) + blocks * Hkv * 8 + T * c["rot"] * 4,
                "flops": T * D * (8 * Hq + 12 * Hkv)}
    seen = [_seen(m, t, c["window"], c["sinks"]) for m, t in zip(n, total)]
    return {"bytes": sum(u for _, u in seen) * Hkv * D * 2 + T * Hq * (D * 4 + 4),
            "flops": 4 * D * Hq * sum(p for p, _ in seen)}


# --------------------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "route":
        x = _randn(g, c["T"], c["E"]) * 1.2
        s["logits"] = x if c["dtype"] == "f32" else x.to(torch.bfloat16)
        s["bias"] = _randn(g, c["E"]) * 0.05 if c["bias"] else None
        if own:
            _bind_route(s)
        return s
    n, total = _lengths(c)
    B, page, Hq, Hkv, D = c["batch"], c["page"], c["Hq"], c["Hkv"], c["D"]
    starts = [0]
    for m in n:
        starts.append(starts[-1] + m)
    T = starts[-1]
    s["cu"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    s["T"], s["q_max"], s["ctx_max"] = T, max(n), max(total)
    width = (max(total) + page - 1) // page
    n_pages = sum((t + page - 1) // page for t in total) + 3
    # pages handed out in random order, as an allocator under load does
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    need = torch.tensor([(t + page - 1) // page for t in total], device=DEV)
    col = torch.arange(width, device=DEV)
    row0 = torch.cumsum(need, 0) - need
    table = order[(row0[:, None] + col).clamp(max=n_pages - 1)]
    s["table"] = torch.where(col < need[:, None], table, torch.zeros_like(table)).contiguous()
    s["n_pages"] = n_pages
    for name in ("k", "v"):
        codes = (_randn(g, n_pages * Hkv * page * D) * 100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
        s[name] = codes.view(n_pages, Hkv, page, D)
        e = torch.randint(-8, -5, (n_pages, Hkv), generator=g, device=DEV)
        s[name + "_scale"] = torch.ldexp(torch.ones(n_pages, Hkv, device=DEV), e)
    if c["op"] == "append":
        # queries, keys and values as one projection leaves them: rows of a joint matrix
        qkv = (_randn(g, T, (Hq + 2 * Hkv) * D) * 1.5).to(torch.bfloat16)
        s["qkv"] = qkv
        s["q_new"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k_new"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v_new"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["gamma_q"] = torch.rand(D, generator=g, device=DEV) + 0.5 if c["norm"] else None
        s["gamma_k"] = torch.rand(D, generator=g, device=DEV) + 0.5 if c["norm"] else None
        half = c["rot"] // 2
        i = torch.arange(half, device=DEV, dtype=torch.float64)
        angle = torch.arange(c["ctx_max"], device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-i / half)
        s["cos_sin"] = torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32).contiguous()
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    else:
        s["q"] = _randn(g, T, Hq, D).to(torch.bfloat16)
        # what lies behind a request's last token was never written: it may read as NaN
        last = s["table"][torch.arange(B, device=DEV), (need - 1)].long()
        past = torch.arange(page, device=DEV) >= (s["kv_len"].long() - (need - 1) * page)[:, None]
        for name in ("k", "v"):
            codes = s[name].view(torch.uint8)
            codes[last] = torch.where(past[:, None, :, None], torch.full_like(codes[last], 0x7F), codes[last])
    if own:
        (_bind_append if c["op"] == "append" else _bind_attend)(s)
    return s


# --------------------------------------------------------------------------- the library's calls

def _bind_route(s):
    """The output buffers and call parameters that a serving loop keeps."""
    from top_routed_expert_gb300 import abi
    c = s["c"]
    s["ids"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device=DEV)
    s["w"] = torch.empty(c["T"], c["k"], dtype=torch.float32, device=DEV)
    s["abi"] = abi
    s["cfg"] = abi.make_route_scores_config(
        c["T"], c["E"], c["k"], n_groups=c["G"], top_groups=c["tg"], group_rank=c["rank"],
        score=abi.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else abi.MOE_SCORE_SOFTMAX,
        logit_dtype=abi.MOE_F32 if c["dtype"] == "f32" else abi.MOE_BF16, renormalise=c["norm"], scale=c["scale"])


def _bind_append(s):
    from top_routed_expert_gb300 import abi
    c = s["c"]
    s["abi"] = abi
    s["cache"] = abi.make_kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    s["cfg"] = abi.make_kv_append_config(
        s["q_new"], s["k_new"], s["v_new"], s["q_out"], batch=c["batch"], rot_dim=c["rot"], n_pos=c["ctx_max"],
        rope_layout=abi.MOE_ROPE_HALF if c["layout"] == "half" else abi.MOE_ROPE_INTERLEAVED, eps=1e-6)


def _bind_attend(s):
    from top_routed_expert_gb300 import abi
    c = s["c"]
    s["abi"] = abi
    s["cache"] = abi.make_kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["T"], c["Hq"], dtype=torch.float32, device=DEV)
    s["cfg"] = abi.make_paged_attention_config(
        s["q"], s["out"], batch=c["batch"], max_q_len=s["q_max"], window=c["window"], n_sink=c["sinks"],
        sm_scale=c["D"] ** -0.5)
    s["ws"] = torch.empty(abi.moe_paged_attention_ws_bytes(s["cfg"], s["cache"]), dtype=torch.uint8, device=DEV)


def run(s):
    op = s["c"]["op"]
    if not own:
        return {"route": _route_plain, "append": _append_plain, "attend": _attend_plain}[op](s)
    abi = s["abi"]
    if op == "route":
        abi.moe_route_scores(s["cfg"], s["logits"], s["bias"], s["ids"], s["w"])
        return {"ids": s["ids"], "w": s["w"]}
    if op == "append":
        abi.moe_kv_append(s["cfg"], s["cache"], s["q_new"], s["k_new"], s["v_new"], s["gamma_q"], s["gamma_k"],
                          s["cos_sin"], None, s["cu"], s["kv_len"], s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    abi.moe_paged_attention(s["cfg"], s["cache"], s["q"], s["cu"], s["kv_len"], s["out"], s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------- plain forms

def _route_plain(s):
    c = s["c"]
    L = s["logits"].float()
    T, E, k, G, tg = c["T"], c["E"], c["k"], c["G"], c["tg"]
    if c["score"] == "sigmoid":
        e = 1.0 / (1.0 + torch.exp(-L))
        score = e
    else:
        e = torch.exp(L - L.amax(1, keepdim=True))
        score = e / e.double().sum(1, keepdim=True).float()
    # without a bias the logits give the order of the scores, free of their rounding
    choice = L if s["bias"] is None else score + s["bias"]
    if G > 1 and tg < G:
        member = (L if c["rank"] == 1 else e) if s["bias"] is None else choice
        top = torch.sort(member.view(T, G, E // G), dim=2, descending=True, stable=True)[0]
        group = top[:, :, 0] if c["rank"] == 1 or E == G else top[:, :, 0] + top[:, :, 1]
        keep = torch.sort(group, dim=1, descending=True, stable=True)[1][:, :tg]
        allowed = torch.zeros(T, G, dtype=torch.bool, device=L.device).scatter_(1, keep, True)
        choice = torch.where(allowed.repeat_interleave(E // G, 1), choice, torch.full_like(choice, -math.inf))
    ids = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    w = score.gather(1, ids)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": w * c["scale"]}


def _norm_rotate(x, gamma, cs, rot, layout):
    """RMS norm over the head and rotation of its first `rot` elements, in 32 bits; x [T, H, D], cs [T, rot/2, 2]."""
    y = x.float()
    if gamma is not None:
        y = y * (1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6)) * gamma
    r, rest = y[..., :rot], y[..., rot:]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _token_rows(s):
    """(request, position in its sequence) of each new token."""
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    return b, t - s["cu"].long()[b] + (s["kv_len"].long() - (s["cu"][1:] - s["cu"][:-1]).long())[b]


def _append_plain(s):
    c = s["c"]
    page, D = c["page"], c["D"]
    _, pos = _token_rows(s)
    cs = s["cos_sin"][pos]
    q = _norm_rotate(s["q_new"], s["gamma_q"], cs, c["rot"], c["layout"]).to(torch.bfloat16)
    rows = {"k": _norm_rotate(s["k_new"], s["gamma_k"], cs, c["rot"], c["layout"]), "v": s["v_new"].float()}
    # every page that gets a token: [request, page, slot]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    start = s["kv_len"].long() - n
    first = start // page
    local = torch.arange((s["q_max"] + page - 2) // page + 1, device=DEV)
    b, p = torch.nonzero((first[:, None] + local) * page < s["kv_len"][:, None], as_tuple=True)
    j = (first[b] + p)[:, None] * page + torch.arange(page, device=DEV)
    new = (j >= start[b][:, None]) & (j < s["kv_len"][b][:, None])
    old = j < start[b][:, None]
    row = (s["cu"][b].long()[:, None] + j - start[b][:, None]).clamp(0, max(0, s["T"] - 1))
    at = s["table"][b, first[b] + p].long()
    out = {"q": q}
    for name in ("k", "v"):
        x = torch.where(new[:, :, None, None], rows[name][row], torch.zeros((), device=DEV)).transpose(1, 2)
        # the smallest power of two, at least 2^-40, that leaves no value over 448 = 0.875 * 2^9
        m, e = torch.frexp(x.abs().amax((2, 3)))
        need = torch.ldexp(torch.ones_like(m), torch.where(m <= 0.875, e - 9, e - 8)).clamp(min=2.0 ** -40)
        had = s[name + "_scale"][at]
        scale = torch.where(old[:, :1], torch.maximum(need, had), need)
        was = s[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
        kept = torch.where(old[:, None, :, None], was * (had / scale)[:, :, None, None], was)
        codes = torch.where(new[:, None, :, None], x / scale[:, :, None, None], kept).to(torch.float8_e4m3fn)
        s[name].view(torch.uint8)[at] = codes.view(torch.uint8)
        s[name + "_scale"][at] = scale
        out[name], out[name + "_scale"] = s[name], s[name + "_scale"]
    return out


def _attend_plain(s):
    c = s["c"]
    B, Hq, Hkv, D, page = c["batch"], c["Hq"], c["Hkv"], c["D"], c["page"]
    at = s["table"].long()
    J = at.shape[1] * page
    j = torch.arange(J, device=DEV)

    def values(name):
        x = s[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s[name + "_scale"][at][..., None, None]
        x = x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, J, D)
        return torch.where((j < s["kv_len"][:, None])[:, None, :, None], x, torch.zeros((), device=DEV))

    n = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(s["q_max"], device=DEV)
    row = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["T"] - 1)
    pos = (s["kv_len"].long() - n)[:, None] + i
    q = s["q"][row].float().view(B, -1, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    scores = torch.matmul(q, values("k").transpose(2, 3)) * D ** -0.5
    see = j <= pos[:, :, None]
    if c["window"]:
        see = see & ((j > pos[:, :, None] - c["window"]) | (j < c["sinks"]))
    scores = scores.view(B, Hkv, -1, Hq // Hkv, J).masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, -1, J), values("v")).view(B, Hkv, -1, Hq // Hkv, D) / total.clamp(min=1e-30)
    lse = (top + torch.log(total)).squeeze(-1)
    tb, _ = _token_rows(s)
    ti = torch.arange(s["T"], device=DEV) - s["cu"].long()[tb]
    return {"out": out[tb, :, ti].reshape(s["T"], Hq, D).to(torch.bfloat16), "lse": lse[tb, :, ti].reshape(s["T"], Hq)}


# --------------------------------------------------------------------------- 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return {"route": _route_exact, "append": _append_exact, "attend": _attend_exact}[c["op"]](s)


def _route_exact(s):
    c = s["c"]
    L = s["logits"].double()
    score = torch.sigmoid(L) if c["score"] == "sigmoid" else torch.softmax(L, 1)
    choice = score if s["bias"] is None else score + s["bias"].double()
    size = c["E"] // c["G"]
    groups = choice.view(-1, c["G"], size).topk(min(c["rank"], size), 2)[0].sum(2)
    best = groups.topk(c["tg"], 1)[1]
    group_of = torch.arange(c["E"], device=DEV) // size
    inside = (best[:, :, None] == group_of).any(1)
    ids = torch.topk(choice.masked_fill(~inside, -math.inf), c["k"], 1)[1]
    w = torch.take_along_dim(score, ids, 1)
    return {"ids": ids.to(torch.int32), "w": c["scale"] * (w / w.sum(1, keepdim=True) if c["norm"] else w)}


def _append_exact(s):
    """Codes are given unrounded, as value over scale: what one rounding to E4M3 may move."""
    c = s["c"]
    page, half = c["page"], c["rot"] // 2
    n, total = _lengths(c)
    table = s["table"].tolist()

    def turned(x, gamma, first):
        x = x.double()
        if gamma is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma.double()
        z = torch.view_as_complex(s["cos_sin"].double())[first:first + x.shape[0], None]
        pairs = x[..., :c["rot"]]
        if c["layout"] == "half":
            w = z * torch.complex(pairs[..., :half], pairs[..., half:])
            w = torch.cat([w.real, w.imag], -1)
        else:
            w = torch.view_as_real(z * torch.view_as_complex(pairs.unflatten(-1, (half, 2)).contiguous())).flatten(-2)
        return torch.cat([w, x[..., c["rot"]:]], -1)

    out = {"q": torch.empty(s["T"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)}
    for name in ("k", "v"):
        out[name], out[name + "_scale"] = s[name].double(), s[name + "_scale"].double()
    row = 0
    for b in range(c["batch"]):
        first, end = total[b] - n[b], total[b]
        at = slice(row, row + n[b])
        row += n[b]
        out["q"][at] = turned(s["q_new"][at], s["gamma_q"], first)
        k, v = turned(s["k_new"][at], s["gamma_k"], first), s["v_new"][at].double()
        for pg in range(first // page, (end - 1) // page + 1):
            lo, hi = max(first, pg * page), min(end, (pg + 1) * page)
            where = table[b][pg]
            for name, x in (("k", k), ("v", v)):
                x = x[lo - first:hi - first].transpose(0, 1)
                amax = x.abs().amax((1, 2))
                scale = torch.exp2(torch.ceil(torch.log2((amax / 448).clamp(min=2.0 ** -40))))
                scale = torch.where((scale > 2.0 ** -40) & (amax <= 224 * scale), scale / 2, scale)  # log2 rounds
                had = out[name + "_scale"][where].clone()
                if lo > pg * page:
                    scale = torch.maximum(scale, had)
                    out[name][where, :, :lo - pg * page] *= (had / scale)[:, None, None]
                out[name][where, :, lo - pg * page:hi - pg * page] = x / scale[:, None, None]
                out[name + "_scale"][where] = scale
    return out


def _attend_exact(s):
    c = s["c"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    n, total = _lengths(c)
    out = torch.empty(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["T"], Hq, dtype=torch.float64, device=DEV)
    row = 0
    for b in range(c["batch"]):
        pages = s["table"][b, :(total[b] + page - 1) // page].long()
        at = slice(row, row + n[b])
        row += n[b]
        p = torch.arange(total[b] - n[b], total[b], device=DEV)[:, None]
        j = torch.arange(total[b], device=DEV)[None]
        hidden = j > p
        if c["window"]:
            hidden |= (p - j >= c["window"]) & (j >= c["sinks"])
        for h in range(Hkv):
            k, v = (torch.cat([s[m][x, h].double() * s[m + "_scale"][x, h].double()[:, None, None]
                               for x in pages.split(4096)]).view(-1, D)[:total[b]] for m in ("k", "v"))
            for g in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                z = (s["q"][at, g].double() @ k.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse[at, g] = torch.logsumexp(z, 1)
                out[at, g] = torch.exp(z - lse[at, g][:, None]) @ v
    return {"out": out, "lse": lse}
