"""The balance loss's gradient where its common factor, dloss * coefficient *
experts / (C S), is beyond binary32's normal numbers but the gradient is not.

Bounds as in test_gpu_ops_balance.py, u = 2^-24 (slopes a less that of the row's
best expert): the shares' errors (2 + 2.5 |x - top| of u for softmax, 9 + 5 |x| for
sigmoid) times the last factor and in the sum over the row, 13 u of that sum's
terms, 4 roundings, for sigmoid (9 + 5 |x|) u of its slope, and half a step; of
numbers below the normal ones half a step of theirs, 2^-150, and a rounding before
it."""
from __future__ import annotations

import numpy as np
import pytest

import ops_step_reference as ref
from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24
SMALL = 2.0 ** -149
LARGEST = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def torch():
    import torch

    torch.cuda.set_device(0)
    return torch


@pytest.fixture(scope="module")
def ops(torch):
    from copy_reduce_snac_amd import operators

    return operators


def host(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [6, 64, 72, 300, 1000])
@pytest.mark.parametrize("size,dloss", [(1e6, 1e-24), (1e6, 1e-27), (2.0, 1e38), (2.0, -3e38)])
def test_far_factors(torch, ops, experts, score, size, dloss, accumulate):
    tokens = 40
    g = np.random.default_rng(experts)
    x = np.clip(g.normal(size=(tokens, experts)) * 1.5, -6, 6)
    x[:, 1] = -np.inf                     # masked: share 0, gradient 0
    x[::3, 2] = 9.0                       # nearly all of the shares
    x[1::3, 3] = -60.0                    # a small share, whose gradient is in range where the others' is not
    ids = g.integers(0, experts, (tokens, 2)).astype(np.int32)
    ids[5] = -1
    load = np.stack([np.floor(g.uniform(0, size, experts)) + 1, g.uniform(0.5, 1, experts) * size / 8]).astype(np.float32)
    logits = torch.from_numpy(x.astype(np.float32)).cuda()
    dx = torch.zeros(tokens, experts, device="cuda") if accumulate else torch.empty(tokens, experts, device="cuda")
    ops.balance_backward(logits, torch.from_numpy(ids).cuda(), torch.from_numpy(load).cuda(), dx, score=score, coefficient=0.5,
                         dloss=torch.full((1,), dloss, device="cuda"), accumulate=accumulate)
    hx, hd = host(logits), float(np.float32(dloss))
    want = ref.balance_backward(hx, ids, load, score, 0.5, hd)
    slope = ref.balance_slope(load, 0.5, hd)
    p = ref.shares(hx, score)
    fin = np.where(np.isinf(hx), 0.0, hx)
    top = hx.max(axis=1, keepdims=True)
    r = np.where(p > 0, 2 + 2.5 * np.abs(fin - top) if score == "softmax" else 9 + 5 * np.abs(fin), 0.0)
    off = p * (r + (p * r).sum(axis=1, keepdims=True) + 1)
    a = slope - np.where(hx == top, slope, 0.0).sum(axis=1, keepdims=True)  # one best expert a row
    dot = (p * a).sum(axis=1, keepdims=True)
    err = off * np.abs(a - dot) + p * ((off * np.abs(a)).sum(axis=1, keepdims=True) + 13 * (p * np.abs(a)).sum(axis=1, keepdims=True)
                                       + np.abs(a - dot)) + 5 * np.abs(want)
    if score == "sigmoid":
        err = err + np.abs(want) * (9 + 5 * np.abs(fin))
    err = U * err + SMALL
    got = host(dx)
    assert (got[:, 1] == 0).all() and (got[5] == 0).all()
    assert not np.isnan(got).any()
    inside = np.abs(want) + err < LARGEST
    assert (np.abs(got - want)[inside] <= err[inside]).all(), np.abs(got - want)[inside].max()
    over = np.abs(want) - err > LARGEST
    assert np.isinf(got[over]).all() and (np.sign(got[over]) == np.sign(want[over])).all()
    if size > 2:
        assert np.abs(want).max() > 1e-39 and inside.all()  # of the reference: 10^6 units of the smallest number


def test_small_shares_with_a_large_factor(torch, ops):
    """Shares of 2^-130 to 2^-136, whose scores are normal numbers, and a factor of 2^130: gradients to a few roundings."""
    experts = 1000
    x = np.zeros((5, experts), np.float32)
    x[:, 3] = -np.arange(83, 88, dtype=np.float32)
    load = np.ones((2, experts), np.float32)
    load[0] = 1 + np.arange(experts) % 5
    ids, dx = torch.zeros(5, 1, dtype=torch.int32, device="cuda"), torch.empty(5, experts, device="cuda")
    dloss = np.float32(3e38)
    ops.balance_backward(torch.from_numpy(x).cuda(), ids, torch.from_numpy(load).cuda(), dx, score="softmax", coefficient=1e4,
                         dloss=torch.full((1,), float(dloss), device="cuda"))
    want = ref.balance_backward(x, np.zeros((5, 1), np.int64), load, "softmax", float(np.float32(1e4)), float(dloss))[:, 3]
    # the share's (2 + 2.5 |x|) u and 2 u of the row's sum; the mean of the differences, up to 4, 16 u of it, of a slope of
    # 1 after it; 5 roundings
    err = U * np.abs(want) * (2 + 2.5 * np.abs(x[:, 3]) + 2 + 16 * 4 + 5)
    got = host(dx)[:, 3]
    assert (want != 0).all() and (np.abs(got - want) <= err).all(), (got, want)
