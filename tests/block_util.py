"""Inputs of the tests of the paged 4-bit cache: ragged batches, small enough
for the oracle's loops."""
import numpy as np
import torch

from oracle import block_oracle as bo
from tests.decode_util import bf16_round
from top_routed_expert_gb300 import abi


class BlockBatch:
    """A cache that requests already use, and their new tokens.

    new, total: new tokens and tokens with them, for each request.  order:
    memory order of a page, "hnd" ([head][token][D]) or "nhd".  Pages are
    handed out in random order; what no request has written holds NaN scales.
    """

    def __init__(self, new, total, Hq=8, Hkv=2, D=128, page=16, order="hnd", seed=0, extra_width=0, spare=2, gk=1.0, gv=0.5):
        rng = np.random.default_rng(seed)
        self.new, self.total, self.Hq, self.Hkv, self.D, self.page = list(new), list(total), Hq, Hkv, D, page
        self.B, self.T, self.gk, self.gv = len(new), int(sum(new)), gk, gv
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_len = np.asarray(total, dtype=np.int32)
        need = [-(-max(t, 0) // page) for t in total]
        self.n_pages = sum(need) + spare
        ids = rng.permutation(self.n_pages)
        self.table = np.full((self.B, max(1, max(need) + extra_width)), -1, dtype=np.int32)
        at = 0
        self.codes, self.scales = {}, {}
        used = np.zeros((self.n_pages, page), dtype=bool)
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
            for j in range(max(total[b], 0)):
                used[self.table[b, j // page], j % page] = True
        for name in ("k", "v"):
            self.codes[name] = rng.integers(0, 256, (self.n_pages, Hkv, page, D // 2), dtype=np.uint8)
            s = rng.integers(0x20, 0x30, (self.n_pages, Hkv, page, D // 16), dtype=np.uint8)   # 1/8 to 1/2
            s[np.broadcast_to(~used[:, None, :, None], s.shape)] = 0x7F
            self.scales[name] = s
        self.q = bf16_round(rng.standard_normal((self.T, Hq, D)))
        self.k = bf16_round(rng.standard_normal((self.T, Hkv, D)) * np.exp(rng.standard_normal((self.T, Hkv, 1))))
        self.v = bf16_round(rng.standard_normal((self.T, Hkv, D)) * np.exp(rng.standard_normal((self.T, Hkv, 1))))
        self.order = order

    def oracle_cache(self):
        return bo.BlockCache(self.codes["k"], self.codes["v"], self.scales["k"], self.scales["v"], self.table, self.gk, self.gv)

    def device(self):
        """The cache on the GPU: its tensors (k, v, k_scale, v_scale, table) and the abi cache."""
        out = []
        for c in (self.codes["k"], self.codes["v"], self.scales["k"], self.scales["v"]):
            c = torch.from_numpy(c).cuda()
            if self.order == "nhd":
                c = c.transpose(1, 2).contiguous().transpose(1, 2)
            out.append(c)
        out.append(torch.from_numpy(self.table).cuda())
        return out, abi.make_blockkv_cache(*out, k_gscale=self.gk, v_gscale=self.gv)

    def lengths(self):
        return torch.from_numpy(self.cu).cuda(), torch.from_numpy(self.kv_len).cuda()

    def vmax(self):
        """The largest size that a value can have."""
        s = self.scales["v"]
        return 6.0 * self.gv * max(float(np.max(bo.decode_e4m3(s[s != 0x7F]), initial=0.0)), 1e-30)


def angles(n, rot):
    i = np.arange(rot // 2)
    a = np.arange(n)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def host(t):
    return t.view(torch.uint8).cpu().contiguous().numpy() if t.element_size() == 1 else t.cpu().numpy()
