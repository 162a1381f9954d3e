"""CPU fp64 oracle of the decoder-step operators: expert selection from
scores, append to the paged 8-bit key/value cache, attention over it.

TEST INFRASTRUCTURE.  Only the tests and the package smoke check may import
this module; the library's own code never does, and it shares no code with
the CUDA path.  Written one token, page and row at a time, from the
definitions in include/route_scores.h and include/paged_kv.h; every function
computes in float64.
"""
from __future__ import annotations

import math

import numpy as np

from .moe_oracle import decode_e4m3, encode_e4m3

MIN_SCALE = 2.0 ** -40


# ------------------------------------------------------------- expert selection

def scores(L, kind: str) -> np.ndarray:
    """sigmoid or softmax of one token's logits; -inf, +inf and NaN count as masked."""
    L = np.array(L, dtype=np.float64)
    L[~(L < math.inf)] = -math.inf
    e = np.zeros_like(L)
    if kind == "sigmoid":
        e[L > -math.inf] = 1.0 / (1.0 + np.exp(-L[L > -math.inf]))
        return e
    if np.all(L == -math.inf):
        return e
    e = np.exp(L - L.max())
    return e / e.sum()


def route_scores(logits, bias, k, n_groups=1, top_groups=1, group_rank=1, kind="softmax", renormalise=True,
                 scale=1.0):
    """(ids [T][k], weights [T][k], choice values [T][E]) of float64 logits."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    size = E // n_groups
    ids = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k))
    choice = np.zeros((T, E))
    for t in range(T):
        s = scores(logits[t], kind)
        masked = ~(logits[t] < math.inf) | (logits[t] == -math.inf)
        c = s.copy() if bias is None else s + np.asarray(bias, dtype=np.float64)
        if bias is not None:
            masked = masked | ~(np.asarray(bias) < math.inf) | (np.asarray(bias) == -math.inf)
        c[masked] = -math.inf
        member = c
        if bias is None and group_rank == 2:
            member = s
        value = []
        for g in range(n_groups):
            best = sorted(member[g * size:(g + 1) * size], reverse=True)[:group_rank]
            value.append(sum(best))
        groups = sorted(range(n_groups), key=lambda g: (-value[g], g))[:top_groups]
        inside = [e for g in sorted(groups) for e in range(g * size, (g + 1) * size)]
        order = sorted(inside, key=lambda e: (-c[e], e))[:k]
        ids[t] = order
        got = np.array([0.0 if masked[e] else s[e] for e in order])
        if renormalise:
            got = got / got.sum() if got.sum() > 0 else got * 0.0
        w[t] = scale * got
        choice[t] = c
    return ids, w, choice


# ------------------------------------------------------------- paged cache

def norm_rotate(x, gamma, cs, layout: str, eps: float) -> np.ndarray:
    """RMS norm over the last axis (gamma None: none), then rotation of its
    first 2 len(cs) elements by the angles whose (cos, sin) are cs [r][2]."""
    y = np.array(x, dtype=np.float64)
    if gamma is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(gamma, dtype=np.float64)
    if cs is None or len(cs) == 0:
        return y
    r = len(cs)
    out = y.copy()
    for i in range(r):
        ia, ib = (i, i + r) if layout == "half" else (2 * i, 2 * i + 1)
        a, b = y[..., ia], y[..., ib]
        out[..., ia] = a * cs[i][0] - b * cs[i][1]
        out[..., ib] = b * cs[i][0] + a * cs[i][1]
    return out


def page_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-40 with amax <= 448 s."""
    s = MIN_SCALE
    while amax > 448.0 * s:
        s *= 2.0
    return s


class Cache:
    """E4M3 codes [n_pages][heads][page][D] (given as uint8, held as the values
    they stand for, before the scale) and scales [n_pages][heads]."""

    def __init__(self, k, v, k_scale, v_scale, table):
        self.codes = {"k": decode_e4m3(np.asarray(k)), "v": decode_e4m3(np.asarray(v))}
        self.scale = {"k": np.array(k_scale, dtype=np.float64), "v": np.array(v_scale, dtype=np.float64)}
        self.table = np.asarray(table)
        self.page = self.codes["k"].shape[2]

    def values(self, which, b, h, n):
        """The first n tokens' values of a request's head, [n][D]."""
        out = []
        for j in range(n):
            p = self.table[b, j // self.page]
            out.append(self.codes[which][p, h, j % self.page] * self.scale[which][p, h])
        return np.array(out).reshape(n, self.codes[which].shape[3])


def kv_append(cache: Cache, q, k, v, gamma_q, gamma_k, cos_sin, positions, cu, kv_len, layout="half", eps=1e-6):
    """Appends in place; returns (q', the unrounded value / scale of every new
    element as {"k", "v"} lists of (page, head, slot, values))."""
    rot = lambda t, pos: None if cos_sin is None else np.asarray(cos_sin, dtype=np.float64)[
        pos if positions is None else positions[t]]
    q_out = None if q is None else np.zeros(np.shape(q))
    exact = {"k": [], "v": []}
    for b in range(len(kv_len)):
        n = cu[b + 1] - cu[b]
        start = kv_len[b] - n
        pages = {}
        for i in range(n):
            t, pos = cu[b] + i, start + i
            if q is not None:
                q_out[t] = norm_rotate(q[t], gamma_q, rot(t, pos), layout, eps)
            pages.setdefault(pos // cache.page, []).append((pos % cache.page, t, pos))
        for pg, tokens in pages.items():
            at = cache.table[b, pg]
            first = tokens[0][0]
            for name, src in (("k", k), ("v", v)):
                for h in range(np.shape(src)[1]):
                    rows = [norm_rotate(src[t][h], gamma_k, rot(t, pos), layout, eps) if name == "k"
                            else np.array(src[t][h], dtype=np.float64) for _, t, pos in tokens]
                    finite = [np.max(np.abs(r[np.isfinite(r)]), initial=0.0) for r in rows]
                    s = page_scale(max(finite))
                    if first > 0:
                        old = cache.scale[name][at, h]
                        if s > old:
                            for slot in range(first):
                                cache.codes[name][at, h, slot] = encode_e4m3(cache.codes[name][at, h, slot] * (old / s))
                        s = max(s, old)
                    cache.scale[name][at, h] = s
                    for (slot, _, _), r in zip(tokens, rows):
                        exact[name].append((at, h, slot, r / s))
                        code = np.where(np.isnan(r), math.nan, np.sign(r) * 448.0)
                        code[np.isfinite(r)] = encode_e4m3(r[np.isfinite(r)] / s)
                        cache.codes[name][at, h, slot] = code
    return q_out, exact


def paged_attention(cache: Cache, q, cu, kv_len, sm_scale, window=0, n_sink=0):
    """(out [T][Hq][D], lse [T][Hq]); rows that see nothing: 0 and -inf."""
    T, Hq, D = np.shape(q)
    Hkv = cache.codes["k"].shape[1]
    group = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -math.inf)
    for b in range(len(kv_len)):
        n, total = cu[b + 1] - cu[b], max(kv_len[b], 0)
        if n == 0:
            continue
        for h in range(Hkv):
            K, V = cache.values("k", b, h, total), cache.values("v", b, h, total)
            for i in range(n):
                p = total - n + i
                see = [j for j in range(total) if j <= p and (window == 0 or j > p - window or j < n_sink)]
                if not see:
                    continue
                for hq in range(h * group, (h + 1) * group):
                    z = sm_scale * (K[see] @ np.asarray(q[cu[b] + i][hq], dtype=np.float64))
                    e = np.exp(z - z.max())
                    out[cu[b] + i, hq] = (e / e.sum()) @ V[see]
                    lse[cu[b] + i, hq] = z.max() + math.log(e.sum())
    return out, lse
