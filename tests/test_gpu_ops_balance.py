"""The balance loss and its gradient on the GPU, against
tests/ops_step_reference.py.

Bounds, u = 2^-24.  A softmax exponential is off by (2 + 2.5 |x - top|) u of
itself (subtraction, its product with log2 e, the hardware's exponential); a
sigmoid's score by (9 + 5 |x|) u (that exponential in numerator and
denominator, a sum, a reciprocal, a product).  With r that figure of a logit, a
share p is off by p (r + sum p r + 1) u.
  load     counts exact; the sum of the shares' errors over the tokens, a
           rounding of the sum
  loss     of the load that the call got: a rounding
  dlogits  p (a - sum p a) with a less that of the row's best expert (exact: a
           difference of counts): the share's error times the last factor, p
           times the errors of p in the sum and 12 u of the sum's terms (4 fused
           multiply-adds, 2 additions, 6 over the lanes), its rounding and the
           difference's, 4 roundings more, (9 + 5 |x|) u for the sigmoid's slope,
           and half a step; accumulated: a rounding of the sum more
"""
from __future__ import annotations

import numpy as np
import pytest

import ops_step_reference as ref
from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24
DT = {"f32": "float32", "bf16": "bfloat16"}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 1e-37
COEFFICIENT = 0.02


@pytest.fixture(scope="module")
def torch():
    import torch

    torch.cuda.set_device(0)
    return torch


@pytest.fixture(scope="module")
def ops(torch):
    from copy_reduce_snac_amd import operators

    return operators


@pytest.fixture(scope="module")
def handle(torch):
    import copy_reduce_snac_amd as snac

    h = snac.snac_init(1)
    yield h
    snac.snac_finalize(h)


def host(t):
    return t.detach().double().cpu().numpy()


def share_errors(x, score):
    """Shares and what each may be off by, in units of u."""
    p = ref.shares(x, score)
    x = np.where(np.isinf(x), 0.0, x)
    top = np.where(p > 0, x, -np.inf).max(axis=1, keepdims=True)
    r = np.where(p > 0, 2 + 2.5 * np.abs(x - np.where(np.isinf(top), 0, top)) if score == "softmax" else 9 + 5 * np.abs(x), 0.0)
    return p, p * (r + (p * r).sum(axis=1, keepdims=True) + 1)


def inputs(torch, tokens, experts, topk, dtype, seed, shift=0):
    g = np.random.default_rng(seed)
    x = g.normal(size=(tokens, experts)) * 1.5 + 0.5 * g.normal(size=experts)
    x[g.random(x.shape) < 0.02] = -np.inf
    ids = np.argsort(-x, axis=1)[:, :topk].astype(np.int64)
    ids[np.take_along_axis(x, ids, axis=1) == -np.inf] = -1
    if tokens > 4:
        ids[1], ids[2, 0] = -1, experts  # a padding token; an id of no expert
        x[3], ids[3] = -np.inf, -1       # a row that is masked as a whole
        ids[4] = ids[4, 0]               # one expert in all slots
    wide = torch.full((tokens + 1, shift + experts + 3), 77.0, dtype=getattr(torch, DT[dtype]), device="cuda")
    logits = wide[:tokens, shift:shift + experts]
    logits.copy_(torch.from_numpy(x.astype(np.float32)))
    return wide, logits, torch.from_numpy(ids.astype(np.int32)).cuda()


# every shape that is compiled, rows of whole units and not, many and few choices
SHAPES = [(1, 1, 1), (1, 8, 2), (5, 3, 2), (64, 16, 16), (130, 17, 4), (509, 60, 4), (77, 64, 6), (300, 72, 20), (1000, 128, 8),
          (333, 129, 3), (20, 256, 32), (4097, 256, 8), (100, 257, 8), (260, 512, 10), (50, 513, 2), (99, 1000, 32), (40, 1024, 5)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,topk", SHAPES)
def test_both_ways(torch, ops, handle, dtype, score, tokens, experts, topk):
    shift = experts % 3
    wide, logits, ids = inputs(torch, tokens, experts, topk, dtype, tokens + experts, shift)
    load = torch.full((2 * experts + 1,), 55.0, device="cuda")
    ops.balance_load(logits, ids, load[:-1].view(2, experts), handle, score=score)
    loss = torch.full((2,), 55.0, device="cuda")
    ops.balance_loss(load[:-1].view(2, experts), loss[:1], coefficient=COEFFICIENT)
    torch.cuda.synchronize()
    assert load[-1] == 55 and loss[1] == 55
    load = load[:-1].view(2, experts)
    hx, hi = host(logits), ids.cpu().numpy()
    want = ref.balance_load(hx, hi, score)
    p, off = share_errors(hx, score)
    some = ref.used(hi, experts).any(axis=1, keepdims=True)
    got = host(load)
    assert np.array_equal(got[0], want[0])
    assert (np.abs(got[1] - want[1]) <= U * ((off * some).sum(axis=0) + want[1]) + TINY).all()
    exact = ref.balance_loss(got, np.float32(COEFFICIENT))
    assert abs(float(loss[0]) - exact) <= 2 * U * exact

    dloss = torch.full((1,), 1.5, device="cuda")
    slope = ref.balance_slope(got, np.float32(COEFFICIENT), 1.5)
    finite = np.where(np.isnan(hx), -np.inf, hx)
    best = np.where(finite == finite.max(axis=1, keepdims=True), slope, -np.inf).max(axis=1, keepdims=True)
    a = slope - best
    want = ref.balance_backward(hx, hi, got, score, np.float32(COEFFICIENT), 1.5)
    dot = (p * a).sum(axis=1, keepdims=True)
    err = off * np.abs(a - dot) + p * ((off * np.abs(a)).sum(axis=1, keepdims=True)
                                       + 13 * (p * np.abs(a)).sum(axis=1, keepdims=True) + np.abs(a - dot)) + 4 * np.abs(want)
    if score == "sigmoid":
        err = err + np.abs(want) * (9 + 5 * np.abs(np.where(np.isinf(hx), 0, hx)))
    err = U * err * some + TINY
    for accumulate in (False, True):
        old = torch.randn(tokens, experts, device="cuda").to(logits.dtype)
        wide_d = torch.full((tokens + 1, experts + 5), 77.0, dtype=logits.dtype, device="cuda")
        dx = wide_d[:tokens, 2:2 + experts]
        dx.copy_(old)
        ops.balance_backward(logits, ids, load, dx, score=score, coefficient=COEFFICIENT, dloss=dloss, accumulate=accumulate)
        torch.cuda.synchronize()
        assert (wide_d[tokens:] == 77).all() and (wide_d[:, :2] == 77).all() and (wide_d[:, 2 + experts:] == 77).all()
        total = want + (host(old) if accumulate else 0.0)
        assert (np.abs(host(dx) - total) <= err + (U + HALF[dtype]) * np.abs(total)).all()
        if accumulate:  # a token that does not count is left as it is
            skipped = torch.from_numpy(~some[:, 0]).cuda()
            assert torch.equal(dx[skipped], old[skipped])
    assert (wide[tokens:] == 77).all()


def test_gradient_without_dloss(torch, ops, handle):
    _, logits, ids = inputs(torch, 40, 24, 3, "f32", 3)
    load = torch.empty(2, 24, device="cuda")
    ops.balance_load(logits, ids, load, handle)
    a, b = torch.empty(40, 24, device="cuda"), torch.empty(40, 24, device="cuda")
    ops.balance_backward(logits, ids, load, a, coefficient=0.5)
    ops.balance_backward(logits, ids, load, b, coefficient=0.5, dloss=torch.ones(1, device="cuda"))
    assert torch.equal(a, b) and float(a.abs().sum()) > 0


@pytest.mark.parametrize("tokens", [0, 1, 16, 17, 256, 257, 8192, 8193, 131072])
def test_many_tokens(torch, ops, handle, tokens):
    """Equal shares add up exactly, over however many tokens."""
    e = 32
    logits = torch.zeros(tokens, e, device="cuda")
    ids = (torch.arange(tokens * 4, device="cuda") % e).to(torch.int32).view(tokens, 4)
    load = torch.full((2, e), 9.0, device="cuda")
    loss = torch.full((1,), 9.0, device="cuda")
    for _ in range(2):  # the scratch of one call does not matter to the next
        ops.balance_load(logits, ids, load, handle)
        ops.balance_loss(load, loss, coefficient=0.25)
    assert torch.equal(load[0], torch.bincount(ids.flatten().long(), minlength=e).float())
    assert torch.equal(load[1], torch.full((e,), tokens / e, device="cuda"))
    assert float(loss) == (0.25 if tokens else 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_far_from_zero(torch, ops, handle, score, dtype):
    """Shares keep their ratios where every score underflows."""
    x = torch.tensor([[-300.0, -301.0, -299.0, -1000.0], [-90.0, -91.0, -90.5, -float("inf")], [500.0, 499.0, 0.0, -500.0],
                      [-3.4e38, -3.4e38, -3.4e38, -float("inf")]], device="cuda").to(getattr(torch, DT[dtype]))
    ids = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    load, dx = torch.empty(2, 4, device="cuda"), torch.empty_like(x)
    for r in range(4):
        ops.balance_load(x[r:r + 1], ids[r:r + 1], load, handle, score=score)
        p, off = share_errors(host(x[r:r + 1]), score)
        if r == 3:  # three equal ones, whatever the bound
            off = np.full_like(p, 4.0)
        assert (np.abs(host(load[1]) - p[0]) <= U * (off[0] + 1) + TINY).all(), r
        ops.balance_backward(x[r:r + 1], ids[r:r + 1], load, dx[r:r + 1], score=score)
        want = ref.balance_backward(host(x[r:r + 1]), [[0]], host(load), score, 1.0, 1.0)
        assert (np.abs(host(dx[r:r + 1]) - want) <= 4 * U * off + HALF[dtype] * np.abs(want) + 1e-5 * U).all(), r


def test_values_that_are_not_finite(torch, ops, handle):
    _, logits, ids = inputs(torch, 64, 40, 2, "f32", 11)
    logits, load, dx = logits.clone(), torch.empty(2, 40, device="cuda"), torch.empty(64, 40, device="cuda")
    logits[1, 7] = float("nan")  # a padding token: no part
    ops.balance_load(logits, ids, load, handle)
    assert not load.isnan().any()
    logits[9, 7] = float("nan")
    ops.balance_load(logits, ids, load, handle, score="sigmoid")
    assert bool(load[1].isnan().all()) and not load[0].isnan().any()
    load[1] = 1.0
    ops.balance_backward(logits, ids, load, dx)
    assert dx.isnan().any(dim=1).nonzero().flatten().tolist() == [9]
    assert bool((dx[1] == 0).all() and (dx[3] == 0).all())


def test_nothing_chosen(torch, ops, handle):
    logits, ids = torch.randn(20, 8, device="cuda"), torch.full((20, 2), -1, dtype=torch.int32, device="cuda")
    load, loss, dx = torch.empty(2, 8, device="cuda"), torch.empty(1, device="cuda"), torch.full((20, 8), 5.0, device="cuda")
    ops.balance_load(logits, ids, load, handle)
    ops.balance_loss(load, loss)
    ops.balance_backward(logits, ids, load, dx)
    assert float(loss) == 0 and bool((load == 0).all() and (dx == 0).all())


def test_loads_of_ranks(torch, ops):
    """Ranks' loads, summed by an all_reduce, are the load of all tokens, and every rank's gradient its part of the whole."""
    import copy_reduce_snac_amd as snac
    from copy_reduce_snac_amd import tensors as coll

    n, t, e = 4, 100, 48
    h = snac.snac_init(n)
    try:
        _, logits, ids = inputs(torch, n * t, e, 4, "f32", 5)
        loads = [torch.empty(2, e, device="cuda") for _ in range(n)]
        for r in range(n):
            ops.balance_load(logits[r * t:(r + 1) * t], ids[r * t:(r + 1) * t], loads[r], h)
        coll.all_reduce(loads, loads, h)
        whole = torch.empty(2, e, device="cuda")
        ops.balance_load(logits, ids, whole, h)
        assert torch.equal(loads[0][0], whole[0]) and all(torch.equal(v, loads[0]) for v in loads)
        # n partial sums of one rounding each, and n - 1 additions
        assert bool(((loads[0][1] - whole[1]).abs() <= 2 * n * U * whole[1]).all())
        parts, dx = torch.empty(n * t, e, device="cuda"), torch.empty(n * t, e, device="cuda")
        for r in range(n):
            s = slice(r * t, (r + 1) * t)
            ops.balance_backward(logits[s], ids[s], loads[0], parts[s])
        ops.balance_backward(logits, ids, loads[0], dx)
        assert torch.equal(parts, dx)
    finally:
        snac.snac_finalize(h)
