"""Inputs of the decoder-step operator tests: ragged batches over a paged
8-bit cache, small enough for the fp64 oracle's loops."""
import numpy as np
import torch

from oracle import decode_oracle as do
from top_routed_expert_gb300 import abi


def bf16_round(x):
    return torch.tensor(np.asarray(x)).to(torch.bfloat16)


class Batch:
    """A cache that requests already use, and their new tokens.

    new, total: new tokens and tokens with them, for each request.  order:
    memory order of a page, "hnd" ([head][token][D]) or "nhd".  Pages are
    handed out in random order; what no request has written holds NaN codes.
    """

    def __init__(self, new, total, Hq=8, Hkv=2, D=128, page=16, order="hnd", seed=0, extra_width=0, spare=2):
        rng = np.random.default_rng(seed)
        self.new, self.total, self.Hq, self.Hkv, self.D, self.page = list(new), list(total), Hq, Hkv, D, page
        self.B, self.T = len(new), int(sum(new))
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_len = np.asarray(total, dtype=np.int32)
        need = [-(-max(t, 0) // page) for t in total]
        self.n_pages = sum(need) + spare
        ids = rng.permutation(self.n_pages)
        self.table = np.full((self.B, max(1, max(need) + extra_width)), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (self.n_pages, Hkv, page, D)
        self.codes, self.scales = {}, {}
        for name in ("k", "v"):
            c = np.full(shape, 0x7F, dtype=np.uint8)
            for b, t in enumerate(total):
                for j in range(max(t, 0)):
                    v = torch.tensor(rng.standard_normal((Hkv, D)) * 60.0).clamp(-448, 448).to(torch.float8_e4m3fn)
                    c[self.table[b, j // page], :, j % page] = v.view(torch.uint8).numpy()
            self.codes[name] = c
            self.scales[name] = 2.0 ** rng.integers(-8, -4, (self.n_pages, Hkv))
        self.q = bf16_round(rng.standard_normal((self.T, Hq, D)) * 2.0)
        self.k = bf16_round(rng.standard_normal((self.T, Hkv, D)) * np.exp(rng.standard_normal((self.T, Hkv, 1))))
        self.v = bf16_round(rng.standard_normal((self.T, Hkv, D)) * np.exp(rng.standard_normal((self.T, Hkv, 1))))
        self.order = order
        self.rng = rng

    def oracle_cache(self):
        return do.Cache(self.codes["k"], self.codes["v"], self.scales["k"], self.scales["v"], self.table)

    def device(self):
        """The cache on the GPU as (codes k, v; scales; table; abi cache)."""
        out = []
        for name in ("k", "v"):
            c = torch.from_numpy(self.codes[name]).cuda()
            if self.order == "nhd":
                c = c.transpose(1, 2).contiguous().transpose(1, 2)
            out.append(c.view(torch.float8_e4m3fn))
        sc = [torch.from_numpy(self.scales[n].astype(np.float32)).cuda() for n in ("k", "v")]
        table = torch.from_numpy(self.table).cuda()
        return out[0], out[1], sc[0], sc[1], table, abi.make_kv_cache(out[0], out[1], sc[0], sc[1], table)

    def lengths(self):
        return torch.from_numpy(self.cu).cuda(), torch.from_numpy(self.kv_len).cuda()


def values64(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def codes_of(t):
    """Code bytes of a cache tensor in [page][head][token][D] order."""
    return t.view(torch.uint8).cpu().contiguous().numpy()
