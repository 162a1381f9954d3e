"""GPU parity of moe_add_rms_norm (include/add_rms_norm.h) against fp64.

h: one rounding of the sum to the residual's type, 2^-8 of its size for bf16
(2^-24 for fp32, and the fp32 addition's 2^-24 before).  y, on the h that the
GPU stored: a row's fp32 sum of squares is off by at most (d / threads + 20)
2^-24, the root and three products by 2^-23 more: 1e-5 of |y| is allowed
(16384 elements: 32 a thread), and the output's own rounding (bf16 2^-8).
Scales: those of the largest |y|, 1e-5.  E4M3 codes: half a step, 2^-4 of the
size (2^-10 under the normal range), and 1e-5 of it for y and the scale."""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from top_routed_expert_gb300 import abi

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -23}


def run(x, res, gamma, out=BF16, group=None, total=True, eps=1e-6, stream=None):
    T, d = x.shape
    o = None if out is None else torch.full((T, d), 5.0, dtype=out, device="cuda")
    o8 = None if group is None else torch.full((T, d), 3.0, device="cuda").to(torch.float8_e4m3fn)
    s8 = None if group is None else torch.full((T, d // group if group else 1), 7.0, device="cuda")
    s = None if res is None or not total else torch.full(res.shape, 5.0, dtype=res.dtype, device="cuda")
    cfg = abi.make_add_rms_norm_config(x, res, o, o8, s, group=group or 0, eps=eps)
    torch.cuda.synchronize()
    abi.moe_add_rms_norm(cfg, x, res, gamma, o, o8, s8, s, stream=stream)
    torch.cuda.synchronize()
    return o, o8, s8, s


def f64(t):
    return t.detach().double().cpu().numpy()


def check(x, res, gamma, got, out=BF16, group=None, eps=1e-6):
    o, o8, s8, s = got
    h = x.double() if res is None else x.double() + res.double()
    if res is not None:
        exact = f64(h)
        h = h.float().to(res.dtype) if s is None else s
        assert np.all(np.abs(f64(h) - exact) <= STEP[res.dtype] * np.abs(exact) + 2.0 ** -23 * (np.abs(f64(x)) + np.abs(f64(res))))
    y, _, eight = bo.add_rms_norm(f64(h), None, f64(gamma), eps, group)
    if o is not None:
        assert np.all(np.abs(f64(o) - y) <= (STEP[out] + 1e-5) * np.abs(y))
    if group is not None:
        code, scale = eight
        assert np.all(np.abs(f64(s8) - scale) <= 1e-5 * scale)
        assert np.all(np.abs(f64(o8) - code) <= np.maximum(2.0 ** -4 * np.abs(code), 2.0 ** -10) + 2e-5 * np.abs(code))


def inputs(T, d, x=BF16, res=BF16, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda: torch.randn(T, d, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    return r().to(x).cuda(), None if res is None else (r() * 2).to(res).cuda(), (torch.rand(d, generator=g) + 0.5).cuda()


@pytest.mark.parametrize("T,d", [(1, 8), (3, 16), (5, 24), (2, 1000), (7, 1024), (1, 1032), (2, 2048), (3, 2056), (64, 4096),
                                 (2, 4104), (3, 8192), (1, 8200), (2, 16376), (5, 16384), (1500, 520)])
@pytest.mark.parametrize("x,res,out", [(BF16, BF16, BF16), (F32, BF16, F32), (BF16, F32, BF16), (BF16, None, F32), (F32, None, BF16)])
def test_sizes_and_types(T, d, x, res, out):
    a, r, gamma = inputs(T, d, x, res, seed=T + d)
    check(a, r, gamma, run(a, r, gamma, out), out)
    check(a, r, gamma, run(a, r, gamma, out, 0), out, 0)
    if res is not None:   # the sum is rounded whether it is stored or not
        assert torch.equal(run(a, r, gamma, out, total=False)[0], run(a, r, gamma, out)[0])


@pytest.mark.parametrize("group", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T,blocks", [(1, 1), (3, 3), (33, 7), (2, 31), (5, 32)])
@pytest.mark.parametrize("out", [BF16, None])
def test_groups(group, T, blocks, out):
    x, r, gamma = inputs(T, group * blocks, seed=group + T)
    check(x, r, gamma, run(x, r, gamma, out, group), out, group)


def test_rows_of_zeros_and_of_extreme_sizes():
    x, r, gamma = inputs(6, 512, F32, F32, seed=1)
    x[0], r[0] = 0.0, 0.0
    x[1], r[1] = x[1] * 1e15, r[1] * 1e15
    x[2], r[2] = x[2] * 1e-15, r[2] * 1e-15       # the epsilon's
    x[3, 1:], r[3, 1:] = 0.0, 0.0
    r[4] = -x[4]
    for group in (None, 0, 32):
        got = run(x, r, gamma, F32, group)
        check(x, r, gamma, got, F32, group)
    assert torch.all(run(x, r, gamma, F32, 32)[2][[0, 4]] == 2.0 ** -40)
    check(x, None, gamma, run(x, None, gamma, F32, eps=0.5), F32, eps=0.5)


def test_elements_that_are_not_finite_stay_in_their_row():
    x, r, gamma = inputs(5, 1024, seed=2)
    clean = run(x, r, gamma, F32, 64)
    x[1, 77], x[3, 5] = math.nan, math.inf
    got = run(x, r, gamma, F32, 64)
    for a, b in zip(clean, got):
        assert torch.equal(a[[0, 2, 4]].float(), b[[0, 2, 4]].float())
    assert torch.isnan(got[0][1]).all() and torch.isnan(got[1][1].float()).all()
    assert torch.isnan(got[0][3, 5]) and torch.all(got[0][3, 6:] == 0) and torch.isnan(got[1][3, 5].float())
    assert torch.all(got[2][1] == 2.0 ** -40)


def test_in_place_strided_and_on_another_stream():
    x, r, gamma = inputs(300, 2048, seed=3)
    ref = run(x, r, gamma, BF16, 128)
    a, b = x.clone(), r.clone()                           # the sum over the residual, the norm over x
    cfg = abi.make_add_rms_norm_config(a, b, a, None, b)
    abi.moe_add_rms_norm(cfg, a, b, gamma, a, None, None, b)
    assert torch.equal(a, ref[0]) and torch.equal(b, ref[3])
    a, b = x.clone(), r.clone()                           # the sum over x, the norm over the residual
    cfg = abi.make_add_rms_norm_config(a, b, b, None, a)
    abi.moe_add_rms_norm(cfg, a, b, gamma, b, None, None, a)
    assert torch.equal(b, ref[0]) and torch.equal(a, ref[3])
    wide = [torch.full((300, 2048 + 8 * i), 5.0, dtype=BF16, device="cuda") for i in (1, 3, 2, 5)]
    x2, r2, o2, s2 = (w[:, 8:2056] if i != 0 else w[:, :2048] for i, w in enumerate(wide))
    x2.copy_(x), r2.copy_(r)
    cfg = abi.make_add_rms_norm_config(x2, r2, o2, None, s2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    abi.moe_add_rms_norm(cfg, x2, r2, gamma, o2, None, None, s2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o2, ref[0]) and torch.equal(s2, ref[3])
    assert torch.all(wide[2][:, :8] == 5) and torch.all(wide[3][:, 2056:] == 5)


def test_captured_and_replayed():
    x, r, gamma = inputs(65, 4096, seed=4)
    out, o8, s8, total = torch.empty_like(x), torch.empty(65, 4096, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(65, 1, device="cuda"), torch.empty_like(r)
    cfg = abi.make_add_rms_norm_config(x, r, out, o8, total)
    call = lambda: abi.moe_add_rms_norm(cfg, x, r, gamma, out, o8, s8, total)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    check(x, r, gamma, (out, o8, s8, total), BF16, 0)
