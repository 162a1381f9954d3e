"""Cases, plain forms and 64-bit forms of the operators around a key/value cache held in four bits.

  append  new keys and values into a paged cache of E2M1 codes with an E4M3 scale for every 16 elements; the QK norm
          and the rotation are applied on the way, to the queries as well; the rows written are read back
  attend  attention of the new queries over that cache: causal, grouped heads, optional sliding window with a few first
          tokens that stay visible
  read    rows of the cache as bf16 or fp32
  norm    the residual's addition and the RMS norm behind it, in one pass, with an E4M3 copy and its scales

`own` chooses between the plain torch form and the library's calls."""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# --------------------------------------------------------------------------- cases

def listed():
    return [
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
        # long contexts, what four bits are for: 12 requests of up to 65536 tokens
        dict(name="attend decode 12x65536", op="attend", batch=12, q_len=1, ragged=False, ctx_min=49157,
             ctx_max=65536, Hq=32, Hkv=4, D=128, window=0, sinks=0, page=64),
        # a sliding window with 4 sinks, up to 4 tokens a request (a draft being checked), heads of 64
        dict(name="attend window draft", op="attend", batch=48, q_len=4, ragged=True, ctx_min=5, ctx_max=16381, Hq=32,
             Hkv=8, D=64, window=1024, sinks=4, page=32),
        # chunked prefill: 32 requests, 256 tokens each, over what they have so far
        dict(name="attend prefill 32x256", op="attend", batch=32, q_len=256, ragged=False, ctx_min=256, ctx_max=3584,
             Hq=32, Hkv=4, D=128, window=0, sinks=0, page=16),
        # the whole contexts of a batch, to hand them to another cache or another machine
        dict(name="read 64x3712", op="read", batch=64, q_len=3712, ragged=True, ctx_min=3712, ctx_max=3712, Hkv=4, D=128,
             page=16, dtype="bf16"),
        # the last few tokens of some requests in fp32, as for a look at what was stored
        dict(name="read tails f32", op="read", batch=5, q_len=33, ragged=True, ctx_min=40, ctx_max=701, Hkv=8, D=64,
             page=32, dtype="f32"),
        # a decode batch between attention and experts
        dict(name="norm 64x4096", op="norm", T=64, d=4096, x="bf16", res="bf16", out="bf16", group=-1),
        # a prefill batch, the 8-bit copy for the next projection as well
        dict(name="norm 8192x4096 e4m3", op="norm", T=8192, d=4096, x="bf16", res="bf16", out="bf16", group=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "read", "norm"])
    if op == "norm":
        d = 8 * _log_int(rng, 8, 2048)
        group = rng.choice([-1, 0, 0, 16, 32, 64, 128, 256])
        if group > 0:
            d = max(group, d // group * group)
        return dict(op=op, T=_log_int(rng, 1, min(65536, 2 ** 25 // d)), d=d, x=rng.choice(["bf16", "bf16", "f32"]),
                    res=rng.choice(["bf16", "bf16", "f32", "none"]),
                    out=rng.choice(["bf16", "f32"]) if group < 0 else rng.choice(["bf16", "f32", "none"]), group=group)
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8, 16])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    Hq = Hkv * group
    if op == "read":
        q_len = _log_int(rng, 1, 3712)
        batch = _log_int(rng, 1, min(256, max(1, 2 ** 26 // (q_len * Hkv * D))))
        ctx_max = q_len + _log_int(rng, 1, 2048)
        return dict(op=op, batch=batch, q_len=q_len, ragged=rng.random() < 0.5, ctx_min=rng.randint(q_len, ctx_max),
                    ctx_max=ctx_max, Hkv=Hkv, D=D, page=page, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "append":
        q_len = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2000)
        batch = _log_int(rng, 1, min(256, max(1, 2 ** 25 // (q_len * (Hq + 2 * Hkv) * D))))
        ctx_max = q_len + _log_int(rng, 1, 2048)
        return dict(op=op, batch=batch, q_len=q_len, ragged=rng.random() < 0.5, ctx_min=rng.randint(q_len, ctx_max),
                    ctx_max=ctx_max, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 3 * D // 8]),
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
    """(query, cached token) pairs of a request's n queries; cached tokens that any of them sees."""
    pairs = 0
    for i in range(n):
        p = total - n + i
        pairs += p + 1 if not window or window > p else window + min(sinks, p + 1 - window)
    first = total - n
    union = total if not window or window > first else total - (first - window + 1) + min(sinks, first - window + 1)
    return pairs, union


_SIZE = {"bf16": 2, "f32": 4, "none": 0}
_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_CACHED = 9 / 16   # bytes of a cached element: half a byte of code, a byte of scale for 16


def work(c):
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        eight = T * d + T * (d // c["group"] if c["group"] else 1) * 4 if c["group"] >= 0 else 0
        return {"bytes": T * d * (_SIZE[c["x"]] + 2 * _SIZE[c["res"]] + _SIZE[c["out"]]) + d * 4 + eight,
                "flops": T * d * 6}
    n, total = _lengths(c)
    T, D, Hkv = sum(n), c["D"], c["Hkv"]
    if c["op"] == "read":
        return {"bytes": int(T * Hkv * D * 2 * (_CACHED + _SIZE[c["dtype"]])), "flops": T * Hkv * D * 2}
    Hq = c["Hq"]
    if c["op"] == "append":   # what is read back comes from what was just written, so it counts as written only
        return {"bytes": int(T * (2 * Hq * D * 2 + Hkv * D * 2 * (2 + _CACHED + 2)) + T * c["rot"] * 4),
                "flops": T * D * (8 * Hq + 14 * Hkv)}
    seen = [_seen(m, t, c["window"], c["sinks"]) for m, t in zip(n, total)]
    return {"bytes": int(sum(u for _, u in seen) * Hkv * D * 2 * _CACHED) + T * Hq * (D * 4 + 4),
            "flops": 4 * D * Hq * sum(p for p, _ in seen)}


# --------------------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _normal_codes():
    """Two codes for each of 65536 equally likely numbers: those of normal values whose block is scaled by a third."""
    at = (torch.arange(256, dtype=torch.float64) + 0.5) / 256
    x = torch.erfinv(2 * at - 1) * math.sqrt(2) * 2.9
    limits = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    code = torch.bucketize(x.abs(), limits) + 8 * (x < 0)
    return (code[:, None] + 16 * code[None, :]).flatten().to(torch.uint8).to(DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        s["x"] = (_randn(g, T, d) * 0.7).to(_TYPE[c["x"]])
        # a residual stream: a few channels far larger than the rest
        wide = 1.0 + 30.0 * (torch.rand(d, generator=g, device=DEV) < 0.002)
        s["res"] = None if c["res"] == "none" else (_randn(g, T, d) * wide).to(_TYPE[c["res"]])
        s["gamma"] = torch.rand(d, generator=g, device=DEV) + 0.5
        if own:
            _bind_norm(s)
        return s
    n, total = _lengths(c)
    B, page, Hkv, D = c["batch"], c["page"], c["Hkv"], c["D"]
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
    s["gscale"] = {"k": 1.0, "v": 0.25}
    pairs = _normal_codes()
    last = s["table"][torch.arange(B, device=DEV), (need - 1)].long()
    past = torch.arange(page, device=DEV) >= (s["kv_len"].long() - (need - 1) * page)[:, None]
    for name in ("k", "v"):
        at = torch.randint(0, 65536, (n_pages * Hkv * page * D // 2,), generator=g, device=DEV, dtype=torch.int32)
        s[name] = pairs[at].view(n_pages, Hkv, page, D // 2)
        # scales from 3/16 to 1/2
        e = torch.randint(0x24, 0x30, (n_pages, Hkv, page, D // 16), generator=g, device=DEV, dtype=torch.uint8)
        # what lies behind a request's last token was never written: it may read as NaN
        e[last] = torch.where(past[:, None, :, None], torch.full_like(e[last], 0x7F), e[last])
        s[name + "_scale"] = e.view(torch.float8_e4m3fn)
    if c["op"] == "append":
        Hq = c["Hq"]
        # queries, keys and values as one projection leaves them: rows of a joint matrix
        qkv = (_randn(g, T, (Hq + 2 * Hkv) * D) * 1.5).to(torch.bfloat16)
        s["q_new"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k_new"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v_new"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["gamma_q"] = torch.rand(D, generator=g, device=DEV) + 0.5 if c["norm"] else None
        s["gamma_k"] = torch.rand(D, generator=g, device=DEV) + 0.5 if c["norm"] else None
        half = c["rot"] // 2
        i = torch.arange(half, device=DEV, dtype=torch.float64)
        angle = torch.arange(c["ctx_max"], device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-i / half)
        s["cos_sin"] = torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32).contiguous()
    elif c["op"] == "attend":
        s["q"] = _randn(g, T, c["Hq"], D).to(torch.bfloat16)
    if own:
        {"append": _bind_append, "attend": _bind_attend, "read": _bind_read}[c["op"]](s)
    return s


# --------------------------------------------------------------------------- the library's calls

def _bind_norm(s):
    """The output buffers and call parameters that a serving loop keeps."""
    from top_routed_expert_gb300 import abi
    c, T, d = s["c"], s["c"]["T"], s["c"]["d"]
    s["abi"] = abi
    s["out"] = None if c["out"] == "none" else torch.empty(T, d, dtype=_TYPE[c["out"]], device=DEV)
    s["sum"] = None if s["res"] is None else torch.empty_like(s["res"])
    s["out8"] = s["scale8"] = None
    if c["group"] >= 0:
        s["out8"] = torch.empty(T, d, dtype=torch.float8_e4m3fn, device=DEV)
        s["scale8"] = torch.empty(T, d // c["group"] if c["group"] else 1, dtype=torch.float32, device=DEV)
    s["cfg"] = abi.make_add_rms_norm_config(s["x"], s["res"], s["out"], s["out8"], s["sum"], group=max(0, c["group"]), eps=EPS)


def _bind_cache(s):
    from top_routed_expert_gb300 import abi
    s["abi"] = abi
    s["cache"] = abi.make_blockkv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"],
                                        k_gscale=s["gscale"]["k"], v_gscale=s["gscale"]["v"])


def _bind_read(s):
    _bind_cache(s)
    c = s["c"]
    dtype = _TYPE[c["dtype"]] if c["op"] == "read" else torch.bfloat16
    s["k_rows"], s["v_rows"] = (torch.empty(s["T"], c["Hkv"], c["D"], dtype=dtype, device=DEV) for _ in range(2))
    s["cfg_read"] = s["abi"].make_blockkv_read_config(s["k_rows"], s["v_rows"], batch=c["batch"])


def _bind_append(s):
    _bind_read(s)
    c, abi = s["c"], s["abi"]
    s["q_out"] = torch.empty(s["T"], c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
    s["cfg"] = abi.make_kv_append_config(
        s["q_new"], s["k_new"], s["v_new"], s["q_out"], batch=c["batch"], rot_dim=c["rot"], n_pos=c["ctx_max"],
        rope_layout=abi.MOE_ROPE_HALF if c["layout"] == "half" else abi.MOE_ROPE_INTERLEAVED, eps=EPS)


def _bind_attend(s):
    _bind_cache(s)
    c, abi = s["c"], s["abi"]
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["T"], c["Hq"], dtype=torch.float32, device=DEV)
    s["cfg"] = abi.make_paged_attention_config(
        s["q"], s["out"], batch=c["batch"], max_q_len=s["q_max"], window=c["window"], n_sink=c["sinks"],
        sm_scale=c["D"] ** -0.5)
    s["ws"] = torch.empty(abi.moe_blockkv_attention_ws_bytes(s["cfg"], s["cache"]), dtype=torch.uint8, device=DEV)


def run(s):
    op = s["c"]["op"]
    if not own:
        return {"append": _append_plain, "attend": _attend_plain, "read": _read_plain, "norm": _norm_plain}[op](s)
    abi = s["abi"]
    if op == "norm":
        abi.moe_add_rms_norm(s["cfg"], s["x"], s["res"], s["gamma"], s["out"], s["out8"], s["scale8"], s["sum"])
        return {"out": s["out"], "out8": s["out8"], "scale8": s["scale8"], "sum": s["sum"]}
    if op == "attend":
        abi.moe_blockkv_attention(s["cfg"], s["cache"], s["q"], s["cu"], s["kv_len"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        abi.moe_blockkv_append(s["cfg"], s["cache"], s["q_new"], s["k_new"], s["v_new"], s["gamma_q"], s["gamma_k"],
                               s["cos_sin"], None, s["cu"], s["kv_len"], s["q_out"])
    abi.moe_blockkv_read(s["cfg_read"], s["cache"], s["cu"], s["kv_len"], s["k_rows"], s["v_rows"])
    rows = {"k": s["k_rows"], "v": s["v_rows"]}
    return rows if op == "read" else {"q": s["q_out"], **rows}


# --------------------------------------------------------------------------- plain forms

def _norm_plain(s):
    c = s["c"]
    h = s["x"].float()
    total = None
    if s["res"] is not None:
        total = (h + s["res"].float()).to(s["res"].dtype)
        h = total.float()
    y = h * (1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)) * s["gamma"]
    out8 = scale8 = None
    if c["group"] >= 0:
        z = y.view(c["T"], -1, c["group"] or c["d"])
        scale = (z.abs().amax(2) / 448.0).clamp(min=2.0 ** -40)
        out8 = (z / scale[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(c["T"], c["d"])
        scale8 = scale
    return {"out": None if c["out"] == "none" else y.to(_TYPE[c["out"]]), "out8": out8, "scale8": scale8, "sum": total}


def _tree(x):
    """Sum over the last dimension, a power of two: neighbours first, then their sums."""
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x


def _norm_rotate(x, gamma, cs, rot, layout):
    """RMS norm over the head and rotation of its first `rot` elements in 32 bits; x [T, H, D], cs [T, rot/2, 2].  A key
    that a rounding moves past a code's border is stored as another code, so the order of the sum is that of the
    operator: groups of four, with those that rotate together side by side."""
    y = x.float()
    D = y.shape[-1]
    if gamma is not None:
        four = torch.arange(D // 4, device=DEV)
        if layout == "half" and rot:
            turned = torch.stack([four[:rot // 8], four[rot // 8:rot // 4]], 1).flatten()
            four = torch.cat([turned, four[rot // 4:]])
        squares = (y * y).unflatten(-1, (-1, 4))
        mean = _tree(_tree(squares)[..., 0][..., four]) * (1.0 / D)
        y = y * (1.0 / torch.sqrt(mean + EPS)) * gamma
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


def _values(codes):
    """The values of E2M1 codes [..., n/2 bytes], [..., n]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    both = torch.stack([table[torch.arange(256, device=DEV) % 16], table[torch.arange(256, device=DEV) // 16]], 1)
    return both[codes.int()].flatten(-2)


def _quantise(x, g):
    """(codes, scales) of rows [..., D] whose scales count in units of g."""
    blocks = x.unflatten(-1, (-1, 16))
    top = blocks.abs().amax(-1)
    # the smallest of E4M3's values, at least 2^-9, that leaves no element over 6
    near = (top / 6.0 / g).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    low = (6.0 * near.float() * g < top) & (near.float() < 448.0)
    scale = torch.where(low, near.view(torch.uint8) + 1, near.view(torch.uint8)).view(torch.float8_e4m3fn)
    z = blocks / (scale.float() * g).unsqueeze(-1)
    limits = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    size = z.abs()
    # ties go to the even code: over a limit before an odd one, at or over a limit before an even one
    code = (size > limits[0]).int() + (size >= limits[1]).int() + (size > limits[2]).int() + (size >= limits[3]).int()
    code += (size > limits[4]).int() + (size >= limits[5]).int() + (size > limits[6]).int()
    code = (code + 8 * (z < 0).int()).to(torch.uint8).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scale


def _append_plain(s):
    c = s["c"]
    b, pos = _token_rows(s)
    cs = s["cos_sin"][pos]
    q = _norm_rotate(s["q_new"], s["gamma_q"], cs, c["rot"], c["layout"]).to(torch.bfloat16)
    at, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    k = _norm_rotate(s["k_new"], s["gamma_k"], cs, c["rot"], c["layout"])
    for name, x in (("k", k), ("v", s["v_new"].float())):
        codes, scale = _quantise(x, s["gscale"][name])
        s[name][at, :, slot] = codes
        s[name + "_scale"].view(torch.uint8)[at, :, slot] = scale.view(torch.uint8)
    return {"q": q, **_read_plain(s)}


def _read_plain(s):
    c = s["c"]
    b, pos = _token_rows(s)
    at, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    out = {}
    for name in ("k", "v"):
        scale = s[name + "_scale"].view(torch.uint8)[at, :, slot].view(torch.float8_e4m3fn).float() * s["gscale"][name]
        x = _values(s[name][at, :, slot]).unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)
        out[name] = x.flatten(-2).to(_TYPE[c.get("dtype", "bf16")])
    return out


def _attend_plain(s):
    c = s["c"]
    B, Hq, Hkv, D, page = c["batch"], c["Hq"], c["Hkv"], c["D"], c["page"]
    at = s["table"].long()
    J = at.shape[1] * page
    j = torch.arange(J, device=DEV)

    def values(name):
        scale = s[name + "_scale"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["gscale"][name]
        x = (_values(s[name][at]).unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)).flatten(-2)
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
    return {"append": _append_exact, "attend": _attend_exact, "read": _read_exact, "norm": _norm_exact}[c["op"]](s)


def _norm_exact(s):
    """The 8-bit copy is given unrounded, as value over scale: what one rounding to E4M3 may move."""
    c = s["c"]
    x = s["x"].double()
    total = None
    if s["res"] is not None:
        total = x + s["res"].double()
        # the norm is that of the stored sum; the sum itself is given unrounded
        x = total.float().to(s["res"].dtype).double()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["gamma"].double()
    out8 = scale8 = None
    if c["group"] >= 0:
        parts = y.split(c["group"] or c["d"], 1)
        scale8 = torch.stack([p.abs().max(1).values / 448 for p in parts], 1).clamp(min=2.0 ** -40)
        out8 = y / scale8.repeat_interleave(c["group"] or c["d"], 1)
    return {"out": None if c["out"] == "none" else y, "out8": out8, "scale8": scale8, "sum": total}


def _decoded(s, name, pages, head):
    """Values of one head's pages one after the other, [tokens, D], in 64 bits."""
    byte = s[name][pages, head].flatten(0, 1).long()
    nibble = torch.stack([byte & 15, byte >> 4], -1).flatten(1)
    size = nibble & 7
    x = torch.where(size < 2, size * 0.5, (2.0 + (size & 1)) * torch.exp2((size >> 1).double() - 2.0))
    x = torch.where(nibble > 7, -x, x)
    scale = s[name + "_scale"].view(torch.uint8)[pages, head].flatten(0, 1).view(torch.float8_e4m3fn).double()
    return x * scale.repeat_interleave(16, 1) * s["gscale"][name]


def _read_exact(s):
    c = s["c"]
    n, total = _lengths(c)
    out = {name: torch.empty(s["T"], c["Hkv"], c["D"], dtype=torch.float64, device=DEV) for name in ("k", "v")}
    row = 0
    for b in range(c["batch"]):
        pages = s["table"][b, :(total[b] + c["page"] - 1) // c["page"]].long()
        for name in out:
            for h in range(c["Hkv"]):
                out[name][row:row + n[b], h] = _decoded(s, name, pages, h)[total[b] - n[b]:total[b]]
        row += n[b]
    return out


def _append_exact(s):
    c = s["c"]
    half = c["rot"] // 2
    _, pos = _token_rows(s)

    def turned(x, gamma):
        x = x.double()
        if gamma is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.double()
        z = torch.view_as_complex(s["cos_sin"].double())[pos][:, None]
        pairs = x[..., :c["rot"]]
        if c["layout"] == "half":
            w = z * torch.complex(pairs[..., :half], pairs[..., half:])
            w = torch.cat([w.real, w.imag], -1)
        else:
            w = torch.view_as_real(z * torch.view_as_complex(pairs.unflatten(-1, (half, 2)).contiguous())).flatten(-2)
        return torch.cat([w, x[..., c["rot"]:]], -1)

    steps = torch.arange(1, 127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()   # 2^-9 to 448
    sizes = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)

    def stored(x, g):
        x = x.unflatten(-1, (-1, 16)) / g
        scale = steps[torch.searchsorted(6 * steps, x.abs().amax(-1)).clamp(max=125)].unsqueeze(-1)
        z = (x / scale).abs().clamp(max=6)
        up = torch.searchsorted(sizes, z)
        down = (up - 1).clamp(min=0)
        below, above = z - sizes[down], sizes[up] - z
        pick = torch.where((below < above) | ((below == above) & (down % 2 == 0)), down, up)
        return (torch.sign(x) * sizes[pick] * scale * g).flatten(-2)

    return {"q": turned(s["q_new"], s["gamma_q"]), "k": stored(turned(s["k_new"], s["gamma_k"]), s["gscale"]["k"]),
            "v": stored(s["v_new"].double(), s["gscale"]["v"])}


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
            k, v = (torch.cat([_decoded(s, m, x, h) for x in pages.split(4096)])[:total[b]] for m in ("k", "v"))
            for g in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                z = (s["q"][at, g].double() @ k.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse[at, g] = torch.logsumexp(z, 1)
                out[at, g] = torch.exp(z - lse[at, g][:, None]) @ v
    return {"out": out, "lse": lse}
