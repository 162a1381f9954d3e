"""Scales and codes of moe_blockkv_append (include/block_kv.h) over all that a
bf16 element can be, byte for byte against the oracle, whose quotients and
scales are those of the header's text."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from tests.block_util import BlockBatch
from tests.decode_util import values64
from tests.test_gpu_block_kv import NONFINITE, check_append, check_cache, run_append

pytestmark = pytest.mark.gpu


def of_blocks(blocks, heads, D, seed=0):
    """[n][16] as rows [tokens][heads][D], the last ones filled up with zeros, as bf16; exact."""
    row = heads * D
    flat = np.zeros(-(-blocks.size // row) * row)
    flat[:blocks.size] = blocks.reshape(-1)
    x = torch.from_numpy(flat.reshape(-1, heads, D)).to(torch.bfloat16)
    assert np.array_equal(values64(x), flat.reshape(-1, heads, D))
    return x


def maxima():
    """Sizes in every binade of bf16: its ends, its middle (6 times a power of two is one) and their neighbours."""
    of = np.array([1, 1 + 2.0 ** -7, 1.25, 1.5 - 2.0 ** -7, 1.5, 1.5 + 2.0 ** -7, 1.75, 2 - 2.0 ** -7])
    sizes = torch.from_numpy((of * 2.0 ** np.arange(-133, 128)[:, None]).reshape(-1)).to(torch.bfloat16)
    return np.unique(values64(sizes))


@pytest.mark.parametrize("gk,gv", [(1.0, 2.0 ** -60), (2.0 ** 60, 2.0 ** -9), (2.0 ** -30, 2.0 ** 30)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_block_maxima_of_every_size(gk, gv, layout):
    rng = np.random.default_rng(3)
    top = maxima()
    rest = rng.uniform(-1.0, 1.0, (len(top), 16)) * top[:, None]
    with np.errstate(under="ignore"):
        blocks = values64(torch.from_numpy(rest).to(torch.bfloat16))
    blocks[np.arange(len(top)), rng.integers(0, 16, len(top))] = top * rng.choice([-1.0, 1.0], len(top))
    x = of_blocks(rng.permutation(blocks), 4, 256)
    bt = BlockBatch([len(x)], [len(x) + 3], Hq=1, Hkv=4, D=256, seed=3, gk=gk, gv=gv)
    bt.k.copy_(x)
    bt.v.copy_(x)
    check_append(bt, run_append(bt, layout=layout))


def near_ties(rng, scales):
    """For each scale a block whose first element is 6 of it, the others at the codes' borders or next to them."""
    z = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], (len(scales), 16))
    z *= rng.choice([1.0, 1.0, 1 + 2.0 ** -7, 1 - 2.0 ** -8], z.shape)
    z[:, 0] = 6.0
    return values64(torch.from_numpy(z * scales[:, None] * rng.choice([-1.0, 1.0], z.shape)).to(torch.bfloat16))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_codes_beside_an_infinity(layout):
    """... are the nearest too, ties to the even code."""
    rng = np.random.default_rng(4)
    blocks = near_ties(rng, np.repeat(bo.E4M3_SCALES, 40))
    blocks[np.arange(len(blocks)), rng.integers(1, 16, len(blocks))] = rng.choice([-np.inf, np.inf], len(blocks))
    x = of_blocks(rng.permutation(blocks), 4, 128)
    bt = BlockBatch([len(x)], [len(x) + 3], Hq=1, Hkv=4, D=128, seed=4, gk=1.0, gv=1.0)
    bt.k.copy_(x)
    bt.v.copy_(x)
    r = run_append(bt, layout=layout)
    assert r["st"] == NONFINITE
    ref = bt.oracle_cache()
    _, written = bo.append(ref, None, values64(bt.k), values64(bt.v), None, None, None, None, bt.cu, bt.kv_len)
    check_cache(bt, r, ref, written)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_codes_beside_elements_that_saturate(layout):
    rng = np.random.default_rng(5)
    blocks = near_ties(rng, np.full(2000, 448.0))
    large = rng.choice([-1.0, 1.0], len(blocks)) * 2.0 ** rng.integers(12, 128, len(blocks))
    blocks[np.arange(len(blocks)), rng.integers(1, 16, len(blocks))] = large
    x = of_blocks(blocks, 4, 128)
    bt = BlockBatch([len(x)], [len(x) + 3], Hq=1, Hkv=4, D=128, seed=5, gk=1.0, gv=1.0)
    bt.k.copy_(x)
    bt.v.copy_(x)
    check_append(bt, run_append(bt, layout=layout))
