"""A decoder layer over the paged 8-bit cache: the operators of
include/paged_kv.h and include/route_scores.h with the experts of
include/moe_gb300.h, as a serving loop calls them.

The dense projections (q/k/v, output, router logits) are plain library
products; norms of the residual stream are torch.  Everything between them
runs in the CUDA library.
"""
from __future__ import annotations

from typing import List, Optional

import torch

from . import abi
from .layer import MoELayer


class PagedKVCache:
    """Keys and values of `batch` requests as E4M3 codes in pages, with one
    fp32 scale for each page and key head, and the pages' allocation (on the
    host: a free list and each request's pages in order)."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, batch: int, max_pages: int,
                 device="cuda"):
        self.page_size, self.batch, self.max_pages = page_size, batch, max_pages
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        self.k = torch.empty(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.v = torch.empty(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.k_scale = torch.empty((n_pages, n_kv_heads), dtype=torch.float32, device=device)
        self.v_scale = torch.empty((n_pages, n_kv_heads), dtype=torch.float32, device=device)
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=device)
        self.free: List[int] = list(range(n_pages))
        self.pages: List[List[int]] = [[] for _ in range(batch)]
        self.length = [0] * batch
        self.handle = abi.make_kv_cache(self.k, self.v, self.k_scale, self.v_scale, self.table)

    def extend(self, new: List[int]):
        """Room for new[b] more tokens of each request; returns (cu, kv_len), the two device arrays that the append
        and the attention of those tokens take."""
        if len(new) != self.batch or min(new) < 0:
            raise ValueError("one count of new tokens for each request")
        need = [max(0, -(-(self.length[b] + n) // self.page_size) - len(self.pages[b])) for b, n in enumerate(new)]
        if any(len(self.pages[b]) + n > self.max_pages for b, n in enumerate(need)):
            raise ValueError("a request is longer than the page table is wide")
        if sum(need) > len(self.free):
            raise RuntimeError(f"{sum(need)} pages wanted, {len(self.free)} free")
        for b, n in enumerate(need):
            if n:
                first, got = len(self.pages[b]), self.free[:-n - 1:-1]
                self.table[b, first:first + n] = torch.tensor(got, dtype=torch.int32)
                self.pages[b] += got
                del self.free[-n:]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        length = [have + n for have, n in zip(self.length, new)]
        dev = self.table.device
        arrays = (torch.tensor(cu, dtype=torch.int32, device=dev), torch.tensor(length, dtype=torch.int32, device=dev))
        self.length[:] = length
        return arrays

    def retract(self, new: List[int]):
        """Takes back the last extend(new), whose tokens were not computed.  The pages stay with their requests, which
        will need them again."""
        self.length[:] = [have - n for have, n in zip(self.length, new)]

    def release(self, b: int):
        """Gives request b's pages back."""
        self.free += self.pages[b]
        self.pages[b], self.length[b] = [], 0
        self.table[b] = -1


def rms_norm(x: torch.Tensor, gamma: torch.Tensor, eps: float) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + eps) * gamma).to(torch.bfloat16)


class DecoderLayer:
    """Attention over a PagedKVCache and a mixture of experts, both with a
    residual.  forward() takes the new tokens of all requests at once, prompts
    and single tokens alike.

    w_qkv [(Hq + 2 Hkv) D, d], w_o [d, Hq D] bf16; norm_attn, norm_moe [d];
    gamma_q, gamma_k [D] float32 or None (no QK norm); cos_sin
    [n_pos, rot/2, 2] float32; moe: a MoELayer over bf16 x (its router weights
    and its bias give the logits, as in MoELayer.forward); choice_bias [E]
    float32 or None: added to the scores for the choice alone, the weights stay
    those of the scores (the bias of moe_route_scores); route: further keyword
    arguments of abi.make_route_scores_config.
    """

    def __init__(self, moe: MoELayer, cache: PagedKVCache, w_qkv, w_o, norm_attn, norm_moe, cos_sin, n_q_heads: int,
                 gamma_q=None, gamma_k=None, rope_layout=abi.MOE_ROPE_HALF, window=0, n_sink=0, eps=1e-6,
                 route: Optional[dict] = None, choice_bias: Optional[torch.Tensor] = None):
        self.moe, self.cache, self.w_qkv, self.w_o = moe, cache, w_qkv, w_o
        self.norm_attn, self.norm_moe, self.cos_sin = norm_attn, norm_moe, cos_sin
        self.gamma_q, self.gamma_k = gamma_q, gamma_k
        self.Hq, self.Hkv, self.D = n_q_heads, cache.k.shape[1], cache.k.shape[3]
        self.rope_layout, self.window, self.n_sink, self.eps = rope_layout, window, n_sink, eps
        self.route, self.choice_bias = dict(route or {}), choice_bias
        self._ws = None

    def attention(self, h: torch.Tensor, cu: torch.Tensor, kv_len: torch.Tensor, max_q_len: int) -> torch.Tensor:
        """Attention of the new tokens' states h [T, d] (normed), which it appends to the cache; [T, Hq, D]."""
        T, heads = h.shape[0], (self.Hq, self.Hkv, self.Hkv)
        qkv = h @ self.w_qkv.T
        q, k, v = (x.unflatten(1, (-1, self.D)) for x in qkv.split([n * self.D for n in heads], dim=1))
        q_rot = torch.empty((T, self.Hq, self.D), dtype=torch.bfloat16, device=h.device)
        out = torch.empty_like(q_rot)
        cache = self.cache.handle
        append = abi.make_kv_append_config(q, k, v, q_rot, self.cache.batch, rot_dim=2 * self.cos_sin.shape[1],
                                           n_pos=self.cos_sin.shape[0], rope_layout=self.rope_layout, eps=self.eps)
        abi.moe_kv_append(append, cache, q, k, v, self.gamma_q, self.gamma_k, self.cos_sin, None, cu, kv_len, q_rot)
        attend = abi.make_paged_attention_config(q_rot, out, self.cache.batch, max_q_len=max_q_len, window=self.window,
                                                 n_sink=self.n_sink)
        need = abi.moe_paged_attention_ws_bytes(attend, cache)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=h.device)
        abi.moe_paged_attention(attend, cache, q_rot, cu, kv_len, out, None, self._ws)
        return out

    def choose(self, h: torch.Tensor):
        """(ids, weights) [T, k] of the experts for the states h [T, d]."""
        logits = h.float() @ self.moe.w_router.T
        if self.moe.bias is not None:
            logits += self.moe.bias
        T, k = h.shape[0], self.moe.k
        ids = torch.empty((T, k), dtype=torch.int32, device=h.device)
        w = torch.empty((T, k), dtype=torch.float32, device=h.device)
        abi.moe_route_scores(abi.make_route_scores_config(T, self.moe.E, k, **self.route), logits, self.choice_bias, ids, w)
        return ids, w

    def forward(self, x: torch.Tensor, new: List[int]) -> torch.Tensor:
        """x [T, d] bf16, the states of new[b] more tokens of each request one after the other; the layer's output for
        them.  Pages are handed out on the host, so it runs eagerly; a call that raises leaves the cache's lengths as
        they were, and can be made again."""
        if x.shape[0] != sum(new):
            raise ValueError("as many rows as new tokens")
        cu, kv_len = self.cache.extend(new)
        if x.shape[0] == 0:
            return x
        try:
            a = self.attention(rms_norm(x, self.norm_attn, self.eps), cu, kv_len, max(new))
            x = x + a.flatten(1) @ self.w_o.T
            h = rms_norm(x, self.norm_moe, self.eps)
            return (x.float() + self.moe.forward_routed(h, *self.choose(h)).float()).to(torch.bfloat16)
        except BaseException:
            self.cache.retract(new)
            raise
