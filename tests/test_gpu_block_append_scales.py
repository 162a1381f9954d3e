"""Scales and codes of moe_blockkv_append (include/block_kv.h) over all that a
bf16 element can be, byte for byte against the oracle, whose quotients and
scales are those of the header's text."""
import numpy as np
import pytest
import torch

from tests.block_util import BlockBatch
from tests.decode_util import values64
from tests.test_gpu_block_kv import check_append, run_append

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
