"""Pins of the oracle of the 4-bit cache and of the addition with the norm:
hand-worked values, exhaustive searches and torch, and mistakes planted in the
oracle that a pin has to see."""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from oracle import decode_oracle as do
from oracle import quantize_nvfp4_act_rows


def test_decode_of_every_byte():
    b = np.arange(256, dtype=np.uint8).reshape(1, 1, 16, 16)
    c = bo.BlockCache(b, b, np.full((1, 1, 16, 2), 0x38, np.uint8), np.full((1, 1, 16, 2), 0x40, np.uint8), [[0]], 1.0, 0.25)
    got = c.codes["k"].reshape(256, 2)
    sizes = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for byte in range(256):
        for half, code in enumerate((byte & 15, byte >> 4)):
            assert got[byte, half] == (-1 if code & 8 else 1) * sizes[code & 7]
    assert np.array_equal(c.row("k", 0, 0, 3), c.codes["k"][0, 0, 3])            # scale 1
    assert np.array_equal(c.row("v", 0, 0, 3), c.codes["v"][0, 0, 3] * 0.5)      # scale 2, g 1/4


def pin_block_scale():
    """Against the definition over every code, at and around every border."""
    codes = [float(x) for x in torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()]
    for g in (1.0, 2.0 ** -7, 2.0 ** 20):
        for s in codes:
            for amax in (6 * s * g, 6 * s * g * (1 + 2.0 ** -23), 6 * s * g * (1 - 2.0 ** -23)):
                fits = [c for c in codes if amax <= 6 * c * g]
                assert bo.block_scale(amax, g) == (min(fits) if fits else 448.0)
    assert bo.block_scale(0.0, 1.0) == 2.0 ** -9


def pin_hand_worked_block():
    row = np.zeros(32, dtype=np.float32)
    # largest 6: scale 1; ties to the even code on both sides of 0
    row[:9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -2.5]
    row[9:12] = [-0.75, 2.5000002, 4.9999995]
    # largest 6.5: the smallest scale from 6.5/6 on is 1.125, 6.5/1.125 = 5.78 -> 6
    row[16:19] = [-6.5, 1.0, 0.3]
    values, scales = bo.quantise(row, 1.0)
    assert scales.tolist() == [1.0, 1.125]
    assert values[:12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -2, -1, 3, 4]
    assert values[16:19].tolist() == [-6, 1, 0.5]
    values, scales = bo.quantise(row * 2.0 ** -5, 2.0 ** -5)
    assert scales.tolist() == [1.0, 1.125] and values[16] == -6


def test_block_scale():
    pin_block_scale()


def test_hand_worked_block():
    pin_hand_worked_block()


def test_blocks_are_those_of_the_nvfp4_activations():
    """Where the row scale is g the NVFP4 rounding of activations is the same (its zero blocks apart)."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((20, 64)) * 2.0 ** rng.integers(-3, 3, (20, 1))).astype(np.float32)
    x[:, 0] = 2688.0
    want = quantize_nvfp4_act_rows(x.astype(np.float64))
    for r in range(20):
        v, s = bo.quantise(x[r], 1.0)
        assert np.array_equal(v * np.repeat(s, 16), want[r])


def test_elements_that_are_not_finite():
    row = np.ones(48, dtype=np.float32)
    row[3], row[20], row[21] = math.nan, math.inf, -math.inf
    v, s = bo.quantise(row, 1.0)
    assert math.isnan(s[0]) and s[1] == bo.block_scale(1.0, 1.0) == s[2] and v[20] == 6 and v[21] == -6
    v, s = bo.quantise(np.full(16, 1e30, dtype=np.float32), 1.0)
    assert s[0] == 448 and np.all(v == 6)


def pin_key_rows():
    """The fixed fp32 operations against fp64: a few roundings (2^-24 each) of sums and products, 1e-6 of the largest."""
    rng = np.random.default_rng(2)
    for D, rot, layout in ((64, 64, "half"), (128, 48, "half"), (64, 24, "half"), (256, 256, "interleaved"), (64, 8, "interleaved"),
                           (128, 0, "half")):
        x = torch.tensor(rng.standard_normal(D)).to(torch.bfloat16).double().numpy()
        gamma = rng.uniform(0.5, 1.5, D).astype(np.float32)
        a = rng.uniform(0, 6, rot // 2)
        cs = np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32) if rot else None
        for gm in (gamma, None):
            want = do.norm_rotate(x, gm, cs, layout, 1e-6)
            got = bo.key_rows(x, gm, cs, layout)
            assert np.max(np.abs(got - want)) <= 1e-6 * np.max(np.abs(want))


def test_key_rows():
    pin_key_rows()


def test_order_of_the_sum():
    """1 + 2^-24 + 2^-24: added one after the other the small ones are lost, as neighbours they are not."""
    x = np.zeros(64, dtype=np.float32)
    x[0], x[4], x[5] = 1.0, 2.0 ** -12, 2.0 ** -12          # quads 0 and 1; 2^-24 twice
    one = np.ones(64, dtype=np.float32)
    up = np.float32(1) / np.sqrt(np.float32(1 + 2.0 ** -23) * np.float32(1 / 64) + np.float32(1e-6))
    assert bo.key_rows(x, one, None, "half")[0] == up
    # a rotation of all 64 puts quad 8 beside quad 0
    x[36], x[37], x[4], x[5] = x[4], x[5], 0, 0
    cs = np.tile(np.array([[1.0, 0.0]], dtype=np.float32), (32, 1))
    assert bo.key_rows(x, one, cs, "half")[0] == up


def test_append_and_attention_on_blocks():
    """Values read through the table, attention on them by torch."""
    rng = np.random.default_rng(3)
    table = np.array([[2, 0], [1, 3]])
    z = lambda n: np.zeros((4, 1, 16, n), np.uint8)
    c = bo.BlockCache(z(32), z(32), z(4), z(4), table, 1.0, 0.5)
    k, v, q = (torch.tensor(rng.standard_normal((25, h, 64))).to(torch.bfloat16).double().numpy() for h in (1, 1, 2))
    cu, ln = np.array([0, 20, 25]), np.array([20, 5])
    _, written = bo.append(c, q, k, v, None, None, None, None, cu, ln)
    assert len(written) == 50 and ("k", 0, 0, 3) in written and ("v", 1, 0, 4) in written
    for b in range(2):
        for name, x in (("k", k), ("v", v)):
            got = c.values(name, b, 0, ln[b])
            want = x[cu[b]:cu[b + 1], 0]
            top = np.max(np.abs(want.reshape(ln[b], 4, 16)), -1)     # a scale is at most 9/8 of top / 6, half a step is that
            assert np.all(np.abs(got - want) <= 1.13 / 6 * np.repeat(top, 16, 1))
    out, lse = do.paged_attention(c, q, cu, ln, 0.125)
    K, V = (torch.tensor(c.values(n, 0, 0, 20)) for n in "kv")
    s = torch.tensor(q[:20]).transpose(0, 1) @ K.T * 0.125
    s = s.masked_fill(torch.ones(20, 20).triu(1).bool(), -math.inf)
    assert np.allclose(out[:20], (torch.softmax(s, -1) @ V).transpose(0, 1).numpy(), atol=1e-12)
    assert np.allclose(lse[:20], torch.logsumexp(s, -1).T.numpy(), atol=1e-12)


def pin_add_rms_norm():
    g = torch.Generator().manual_seed(4)
    x, r = torch.randn(5, 96, generator=g).double(), torch.randn(5, 96, generator=g).double()
    gamma = torch.rand(96, generator=g).double()
    y, total, (code, s) = bo.add_rms_norm(x.numpy(), r.numpy(), gamma.numpy(), 1e-3, 32)
    want = torch.nn.functional.rms_norm(x + r, (96,), gamma, 1e-3)
    assert np.allclose(y, want.numpy(), atol=1e-13) and np.allclose(total, (x + r).numpy(), atol=0)
    assert s.shape == (5, 3) and np.allclose(code.reshape(5, 3, 32) * s[..., None], y.reshape(5, 3, 32), atol=1e-13)
    assert np.allclose(np.max(np.abs(code.reshape(5, 3, 32)), -1), 448.0)
    assert bo.add_rms_norm(x.numpy(), None, gamma.numpy(), group=0)[2][1].shape == (5, 1)
    assert np.all(bo.add_rms_norm(np.zeros((1, 16)), None, np.ones(16), group=16)[2][1] == 2.0 ** -40)


def test_add_rms_norm():
    pin_add_rms_norm()


# ----------------------------------------------------------------- mistakes

def off_scale(real):
    return lambda amax, g: max(2.0 ** -9, real(amax, g) / 1.125 if real(amax, g) == 1.125 else real(amax, g))


MISTAKES = [
    ("block_scale", lambda real: lambda amax, g: real(np.nextafter(amax, np.inf), g), pin_block_scale),
    ("block_scale", lambda real: lambda amax, g: real(amax, 1.0), pin_block_scale),
    ("block_scale", off_scale, pin_hand_worked_block),
    ("encode_e2m1", lambda real: lambda v: real(v * (1 + 1e-12)), pin_hand_worked_block),      # ties away from zero
    ("encode_e2m1", lambda real: lambda v: real(v * (1 - 1e-12)), pin_hand_worked_block),      # ... towards it
    ("encode_e2m1", lambda real: lambda v: real(np.abs(v)), pin_hand_worked_block),            # no sign
    ("key_rows", lambda real: lambda x, gm, cs, layout, eps=1e-6: real(x, gm, cs, "interleaved" if layout == "half" else "half", eps),
     pin_key_rows),
    ("key_rows", lambda real: lambda x, gm, cs, layout, eps=1e-6: real(x, gm, None if cs is None else cs * [1, -1], layout, eps),
     pin_key_rows),
    ("key_rows", lambda real: lambda x, gm, cs, layout, eps=1e-6: real(x, gm, cs, layout, 1e-4), pin_key_rows),
    ("add_rms_norm", lambda real: lambda x, r, gm, eps=1e-6, group=None, **kw: real(x, r, gm, eps * 2, group), pin_add_rms_norm),
    ("add_rms_norm", lambda real: lambda x, r, gm, eps=1e-6, group=None, **kw: real(x, None, gm, eps, group), pin_add_rms_norm),
]


@pytest.mark.parametrize("i", range(len(MISTAKES)))
def test_mistakes_are_seen(monkeypatch, i):
    name, mistaken, pin = MISTAKES[i]
    pin()
    monkeypatch.setattr(bo, name, mistaken(getattr(bo, name)))
    with pytest.raises((AssertionError, TypeError)):
        pin()
