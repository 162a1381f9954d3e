"""CPU oracle of the paged 4-bit key/value cache (include/block_kv.h) and of
the residual's addition with the norm behind it (include/add_rms_norm.h).

TEST INFRASTRUCTURE, like decode_oracle, whose attention runs on BlockCache
too.  float64, but for the two places where the header fixes fp32 operations:
a key's norm and rotation before it is quantised (key_rows) and the quotient
that a code is the nearest value of; NumPy's float32 operations are IEEE's.
"""
from __future__ import annotations

import math

import numpy as np

from . import decode_oracle as do
from .moe_oracle import decode_e4m3, encode_e2m1

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3_SCALES = decode_e4m3(np.arange(1, 127, dtype=np.uint8))   # 2^-9 to 448


def block_scale(amax: float, g: float) -> float:
    """The smallest E4M3 value s >= 2^-9 with amax <= 6 s g, 448 where there is none."""
    for s in E4M3_SCALES:
        if amax <= 6.0 * s * g:
            return float(s)
    return 448.0


def quantise(row, g: float):
    """(E2M1 values [n], scales [n / 16]) of a float32 row; a block with a NaN has scale NaN."""
    row = np.asarray(row, dtype=np.float32)
    values, scales = np.zeros(len(row)), np.zeros(len(row) // 16)
    for i in range(len(scales)):
        x = row[16 * i:16 * i + 16]
        if np.isnan(x).any():
            scales[i] = math.nan
            continue
        fine = np.isfinite(x)
        s = block_scale(float(np.max(np.abs(x[fine]), initial=0.0)), g)
        z = np.sign(x) * 6.0
        with np.errstate(over="ignore"):
            z[fine] = encode_e2m1(np.clip((x[fine] / np.float32(s * g)).astype(np.float64), -6, 6))
        values[16 * i:16 * i + 16], scales[i] = z, s
    return values, scales


def key_rows(x, gamma, cs, layout: str, eps: float = 1e-6) -> np.ndarray:
    """Norm and rotation of one row [D] in fp32, operation by operation in the header's order."""
    f = np.float32
    x = np.asarray(x, dtype=f)
    D, r = len(x), 0 if cs is None else len(cs)
    y = x.copy()
    with np.errstate(all="ignore"):
        if gamma is not None:
            four = [(x[i] * x[i] + x[i + 1] * x[i + 1]) + (x[i + 2] * x[i + 2] + x[i + 3] * x[i + 3]) for i in range(0, D, 4)]
            order = list(range(D // 4))
            if layout == "half" and r:
                turned = [q for i in range(r // 4) for q in (i, r // 4 + i)]
                order = turned + order[r // 2:]
            sums = [four[q] for q in order]
            while len(sums) > 1:
                sums = [sums[i] + sums[i + 1] for i in range(0, len(sums), 2)]
            rstd = f(1) / np.sqrt(sums[0] * f(1.0 / D) + f(eps))
            y = (x * rstd) * np.asarray(gamma, dtype=f)
        out = y.copy()
        for i in range(r):
            ia, ib = (i, i + r) if layout == "half" else (2 * i, 2 * i + 1)
            c, s = f(cs[i][0]), f(cs[i][1])
            out[ia] = y[ia] * c - y[ib] * s
            out[ib] = y[ib] * c + y[ia] * s
    return out


class BlockCache:
    """E2M1 codes [n_pages][heads][page][D/2] and E4M3 scales [n_pages][heads][page][D/16] as bytes; codes are held as
    the values they stand for, before the scale."""

    def __init__(self, k, v, k_scale, v_scale, table, gk=1.0, gv=1.0):
        def decode(b):
            b = np.asarray(b).astype(np.int64)
            both = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)
            return np.where(both > 7, -1.0, 1.0) * E2M1[both & 7]
        self.codes = {"k": decode(k), "v": decode(v)}
        self.scale = {"k": decode_e4m3(np.asarray(k_scale)), "v": decode_e4m3(np.asarray(v_scale))}
        self.g = {"k": gk, "v": gv}
        self.table = np.asarray(table)
        self.page = self.codes["k"].shape[2]

    def row(self, which, page, h, slot):
        return self.codes[which][page, h, slot] * np.repeat(self.scale[which][page, h, slot], 16) * self.g[which]

    def values(self, which, b, h, n):
        """The first n tokens' values of a request's head, [n][D]."""
        D = self.codes[which].shape[3]
        return np.array([self.row(which, self.table[b, j // self.page], h, j % self.page) for j in range(n)]).reshape(n, D)


def append(cache: BlockCache, q, k, v, gamma_q, gamma_k, cos_sin, positions, cu, kv_len, layout="half", eps=1e-6):
    """Appends in place; returns (q' in fp64, list of (name, page, head, slot) that were written)."""
    q_out = None if q is None else np.zeros(np.shape(q))
    written = []
    for b in range(len(kv_len)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            t, pos = cu[b] + i, kv_len[b] - n + i
            cs = None if cos_sin is None else np.asarray(cos_sin)[pos if positions is None else positions[t]]
            if q is not None:
                q_out[t] = do.norm_rotate(q[t], gamma_q, cs, layout, eps)
            page, slot = cache.table[b, pos // cache.page], pos % cache.page
            for h in range(np.shape(k)[1]):
                for name, row in (("k", key_rows(k[t][h], gamma_k, cs, layout, eps)), ("v", v[t][h])):
                    cache.codes[name][page, h, slot], cache.scale[name][page, h, slot] = quantise(row, cache.g[name])
                    written.append((name, page, h, slot))
    return q_out, written


def add_rms_norm(x, residual, gamma, eps=1e-6, group=None, rounded=lambda h: h):
    """(y, sum, (codes before rounding, scales) or None); rounded: to the residual's type."""
    h = np.asarray(x, dtype=np.float64)
    total = None
    if residual is not None:
        total = h = rounded(h + np.asarray(residual, dtype=np.float64))
    y = h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps) * np.asarray(gamma, dtype=np.float64)
    eight = None
    if group is not None:
        z = y.reshape(len(y), -1, group or y.shape[1])
        s = np.maximum(np.max(np.abs(z), -1) / 448.0, 2.0 ** -40)
        eight = (z / s[:, :, None]).reshape(y.shape), s
    return y, total, eight


