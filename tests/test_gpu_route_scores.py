"""GPU parity of moe_route_scores (include/route_scores.h) against the fp64
oracle.

The choice is made on fp32 scores plus a bias: expf within 2 ulp, a division
and up to two sums leave an error of at most about 6e-7 on values of size 1 to
2, so two experts or groups whose fp64 values lie within 2e-6 may swap; a token
without such a pair has to be equal.  A weight is a quotient of such scores and
their sum: 2e-6 relative is allowed (a few roundings of 2^-24, expf's 2 ulp)."""
import math

import numpy as np
import pytest
import torch

from oracle import decode_oracle as do
from top_routed_expert_gb300 import abi

pytestmark = pytest.mark.gpu

NEAR = 2e-6
WREL = 2e-6


def run(L, bias, k, G=1, tg=1, rank=1, kind="softmax", renorm=True, scale=1.0, gap=0, stream=None):
    """L: a torch tensor [T, E] (f32 or bf16); gap: elements between rows."""
    T, E = L.shape
    x = torch.full((T, E + gap), 1e30, dtype=L.dtype, device="cuda")
    x[:, :E] = L.cuda()
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    cfg = abi.make_route_scores_config(T, E, k, G, tg, rank,
                                       abi.MOE_SCORE_SIGMOID if kind == "sigmoid" else abi.MOE_SCORE_SOFTMAX,
                                       abi.MOE_F32 if L.dtype == torch.float32 else abi.MOE_BF16, renorm, scale, E + gap)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, dtype=np.float32)).cuda()
    torch.cuda.synchronize()
    abi.moe_route_scores(cfg, x, b, ids, w, stream=stream)
    st = abi.moe_get_device_status(stream)
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64), st


def near(choice, member, k, G, tg, rank):
    """Whether a token's choice hangs on values within NEAR of each other."""
    E = len(choice)
    size = E // G
    if tg < G:
        val = np.array([np.sort(member[g * size:(g + 1) * size])[::-1][:rank].sum() for g in range(G)])
        s = np.sort(val)[::-1]
        if s[tg - 1] - s[tg] < NEAR:
            return True
        keep = np.argsort(-val, kind="stable")[:tg]
        choice = np.concatenate([choice[g * size:(g + 1) * size] for g in keep])
    s = np.sort(choice)[::-1][:k + 1]
    return bool(np.any(s[:-1] - s[1:] < NEAR))


CASES = [
    # T, E, k, G, tg, rank, kind, bias, renorm, scale
    (1, 128, 6, 1, 1, 1, "softmax", False, True, 1.0),
    (64, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5),
    (33, 256, 8, 8, 3, 1, "softmax", False, True, 1.0),
    (33, 256, 16, 32, 7, 2, "softmax", True, False, 1.5),
    (129, 160, 6, 8, 3, 1, "softmax", False, False, 16.0),
    (70, 72, 5, 3, 2, 2, "sigmoid", False, True, 1.0),
    (35, 60, 4, 1, 1, 1, "softmax", True, True, 1.0),
    (19, 8, 8, 1, 1, 2, "sigmoid", True, True, 1.0),
    (7, 1, 1, 1, 1, 1, "softmax", False, False, 1.0),
    (50, 64, 2, 32, 1, 2, "sigmoid", False, False, 1.0),
    (21, 250, 9, 25, 5, 2, "sigmoid", True, True, 1.0),
    (40, 33, 16, 3, 2, 2, "softmax", False, True, 1.0),
    (40, 32, 16, 32, 20, 2, "sigmoid", True, True, 1.0),
]


@pytest.mark.parametrize("T,E,k,G,tg,rank,kind,bias,renorm,scale", CASES)
@pytest.mark.parametrize("dtype,gap", [(torch.float32, 0), (torch.bfloat16, 5), (torch.float32, 3)])
def test_shapes(T, E, k, G, tg, rank, kind, bias, renorm, scale, dtype, gap):
    rng = np.random.default_rng(T * 7 + E)
    L = torch.from_numpy(rng.standard_normal((T, E)) * 1.5).to(dtype)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    ids, w, st = run(L, b, k, G, tg, rank, kind, renorm, scale, gap)
    assert st == 0
    x = L.double().numpy()
    ref_ids, ref_w, choice = do.route_scores(x, b, k, G, tg, rank, kind, renorm, scale)
    clean = 0
    for t in range(T):
        assert len(set(ids[t])) == k and ids[t].min() >= 0 and ids[t].max() < E
        member = choice[t] if b is not None or rank == 1 else do.scores(x[t], kind)
        if near(choice[t], member, k, G, tg, rank) and dtype == torch.float32:
            continue
        if near(choice[t], member, k, G, tg, rank) and not np.array_equal(ids[t], ref_ids[t]):
            continue
        clean += 1
        assert np.array_equal(ids[t], ref_ids[t]), t
        assert np.all(np.abs(w[t] - ref_w[t]) <= WREL * np.abs(ref_w[t])), t
    assert clean > 0.9 * T


@pytest.mark.parametrize("kind,rank,bias", [("softmax", 1, False), ("sigmoid", 1, False), ("sigmoid", 2, True),
                                            ("softmax", 2, False)])
@pytest.mark.parametrize("E,G,tg,k", [(128, 1, 1, 8), (256, 8, 4, 8), (72, 9, 3, 6)])
def test_exact_ties_go_to_the_lowest_index(kind, rank, bias, E, G, tg, k):
    rng = np.random.default_rng(E + k)
    L = torch.from_numpy(rng.integers(-2, 2, (200, E)) * 0.5).float()   # few distinct values
    L[0] = 0.0
    b = np.zeros(E, dtype=np.float32) if bias else None
    ids, w, st = run(L, b, k, G, tg, rank, kind)
    ref_ids, ref_w, _ = do.route_scores(L.numpy(), b, k, G, tg, rank, kind)
    assert st == 0 and np.array_equal(ids, ref_ids)
    assert np.array_equal(ids[0], np.arange(k))
    assert np.all(np.abs(w - ref_w) <= WREL)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("G,tg", [(1, 1), (4, 2)])
def test_masked_experts(kind, bias, G, tg):
    rng = np.random.default_rng(5)
    T, E, k = 12, 64, 6
    L = torch.from_numpy(rng.standard_normal((T, E))).float()
    L[0] = -math.inf                                  # nothing left
    L[1, 3:] = -math.inf                              # fewer than k left
    L[2, ::2] = -math.inf
    L[3, 5] = -math.inf
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    if bias:
        b[7] = -math.inf                              # out of the choice
    ids, w, st = run(L, b, k, G, tg, 1, kind)
    assert st == 0                                    # a mask is no fault
    ref_ids, ref_w, _ = do.route_scores(L.numpy(), b, k, G, tg, 1, kind)
    assert np.array_equal(ids, ref_ids) and np.all(np.abs(w - ref_w) <= WREL)
    assert np.all(w[0] == 0.0) and np.all(w[1, 3:] == 0.0)
    if G == 1:
        assert np.array_equal(ids[0], np.arange(k))


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_nonfinite_logits_are_masked_and_reported(value):
    rng = np.random.default_rng(6)
    L = torch.from_numpy(rng.standard_normal((9, 128))).float()
    ref, ref_w, _ = run(L, None, 6)
    L[4, 17] = value
    ids, w, st = run(L, None, 6)
    assert st == 8                                    # MOE_ERR_DEVICE_NONFINITE
    assert abi.moe_get_device_status() == 0
    keep = np.arange(9) != 4
    assert np.array_equal(ids[keep], ref[keep]) and np.array_equal(w[keep], ref_w[keep])
    masked = L.clone()
    masked[4, 17] = -math.inf
    same, same_w, _ = run(masked, None, 6)
    assert np.array_equal(ids, same) and np.array_equal(w, same_w) and 17 not in ids[4]


def test_peaked_logits_keep_their_order():
    """Without a bias the logits' order decides, also where the scores underflow or saturate."""
    L = torch.from_numpy(np.linspace(-300.0, 300.0, 128)[None].repeat(3, 0)).float()
    for kind in ("softmax", "sigmoid"):
        ids, w, st = run(L, None, 10, kind=kind)
        assert st == 0 and np.array_equal(ids[0], np.arange(127, 117, -1))
        assert np.all(np.isfinite(w))


def test_long_batch_and_other_stream():
    g = torch.Generator().manual_seed(7)
    L = torch.randn(40001, 256, generator=g)
    b = torch.randn(256, generator=g).numpy() * 0.05
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ids, w, st = run(L, b, 8, 8, 4, 2, "sigmoid", True, 2.5, stream=s)
    assert st == 0
    part, part_w, _ = run(L[-37:], b, 8, 8, 4, 2, "sigmoid", True, 2.5)
    assert np.array_equal(ids[-37:], part) and np.array_equal(w[-37:], part_w)
    assert np.all(np.abs(w.sum(1) - 2.5) <= 1e-5)


def test_feeds_the_permutation():
    """ids of a grouped choice go through moe_permute as moe_route's do."""
    T, E, k = 50, 128, 6
    L = torch.randn(T, E, generator=torch.Generator().manual_seed(8))
    cfg = abi.make_config(T, 256, E, k, 64, 64)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    abi.moe_route_scores(abi.make_route_scores_config(T, E, k, 8, 4, 2, abi.MOE_SCORE_SIGMOID), L.cuda(), None, ids, w)
    offs = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    sp, row = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(abi.moe_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_permute(cfg, ids, offs, sp, row, ws)
    assert abi.moe_get_device_status() == 0
    assert torch.equal(torch.bincount(ids.flatten().long(), minlength=E).cumsum(0).int(), offs[1:])
