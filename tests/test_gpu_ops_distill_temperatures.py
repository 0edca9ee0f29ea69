"""The loss against a teacher's top logits at the ends of the accepted
temperatures, whole and in shards, values against tests/ops_step_reference.py.

Bounds, u = 2^-24, as test_gpu_ops_distill.py derives them: an exponential of
arg = (x - top) / temperature is off by (2 + 2.5 |arg|) u of itself.
  S     the terms' errors, and 8 u of the sum; a rounding more for a shard's part
        and one for the joint sum
  q     q (r + sum q r + 2) u with r = 2 + 2.5 |arg|
  loss  sum of q's errors times |log q - log p| + 1, S's and the teacher's sum's
        relative errors, a rounding; joined from shards a rounding of each
        part's D (its size) and Q (times the distance of the shard's maximum)
  dz    |factor| u (p (r + 4) + q's error + 3 q) and half a step
An exponential below binary32's normal numbers, 2^-126, is 0: 2^-126 of a share.
"""
from __future__ import annotations

import numpy as np
import pytest

import ops_step_reference as ref
from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}
TINY = 1e-37


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


def error(arg):
    return 2 + 2.5 * np.abs(arg)


def inputs(torch, dtype, seed, tokens=16, vocab=700, topk=9):
    """Logits with ties at the top in some rows, padding and masked ones."""
    g = np.random.default_rng(seed)
    z, t = g.normal(size=(tokens, vocab)), 2.0 + 2 * g.normal(size=(tokens, topk))
    ids = np.argsort(g.random((tokens, vocab)), axis=1)[:, :topk].astype(np.int64)
    for r in range(tokens):
        z[r, ids[r]] = t[r] + 0.5 * g.normal(size=topk)
    z[1, [3, 400]] = z[1].max() + 1   # two largest logits
    t[2, [0, 5]] = t[2].max() + 1     # two largest of the teacher
    ids[3], ids[4, 0], t[5, 1] = -1, vocab, -np.inf
    z[6, 50:60] = np.where(np.isin(np.arange(50, 60), ids[6]), z[6, 50:60], -np.inf)
    z = torch.from_numpy(z.astype(np.float32)).to(getattr(torch, dtype)).cuda()
    return z, torch.from_numpy(ids).cuda(), torch.from_numpy(t.astype(np.float32)).cuda()


def bounds(z, ids, t, tau, loss):
    """Bounds of loss and S and, for the gradient, the teacher's part."""
    q, logq, ok = ref.choices(ids, t, z.shape[1], tau)
    r = error(np.where(q > 0, logq - logq.max(axis=1, keepdims=True, where=ok, initial=-1e30), 0.0))
    rel = (q * r).sum(axis=1, keepdims=True)
    m = z.max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        arg = np.where(z == -np.inf, 0.0, (z - m) / tau)
        e = np.where(z == -np.inf, 0.0, np.exp(arg))
        s = e.sum(axis=1, keepdims=True)
        s_rel = (e * error(arg)).sum(axis=1, keepdims=True) / s + 8
        logp = np.take_along_axis((z - m) / tau - np.log(s), np.where(ok, ids, 0), axis=1)
        gap = np.where(q > 0, np.abs(logq - logp), 0.0)
    q_off = q * (r + rel + 2)
    return U * ((q_off * (gap + 1)).sum(axis=1) + s_rel[:, 0] + rel[:, 0] + np.abs(loss)) + TINY, U * (s_rel[:, 0] + 1) * s[:, 0], q, q_off, ok


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("tau", [2.0 ** -64, 2.0 ** -30, 1e-4, 0.01, 30.0, 2.0 ** 30, 2.0 ** 64])
def test_values(torch, ops, tau, dtype):
    z, ids, t = inputs(torch, dtype, 5)
    tokens, vocab = z.shape
    loss, stats, dz = torch.empty(tokens, device="cuda"), torch.empty(tokens, 2, device="cuda"), torch.empty_like(z)
    ops.distill(z, ids, t, loss, stats, temperature=tau)
    ops.distill_backward(z, ids, t, stats, dz, temperature=tau, scale=tau)
    tau32 = float(np.float32(tau))
    hz, hi, ht = host(z), ids.cpu().numpy(), host(t)
    want, m, s = ref.distill(hz, hi, ht, tau32)
    off, s_off, q, q_off, ok = bounds(hz, hi, ht, tau32, want)
    assert np.array_equal(host(stats[:, 0]), m)
    assert (np.abs(host(stats[:, 1]) - s) <= s_off).all()
    assert (np.abs(host(loss) - want) <= off).all(), (host(loss), want)
    if tau < 1e-3:  # what the loss is made of: the distance of the teacher's choice from the top
        assert want.max() > 1000 and (host(stats[:, 1]) >= 1).all()

    hs = host(stats)
    back = ref.distill_backward(hz, hi, ht, tau32, hs, np.full(tokens, tau32))
    with np.errstate(all="ignore"):
        arg = np.where(np.isinf(hz), 0.0, (hz - hs[:, :1]) / tau32)
        err = np.where(np.isinf(hz), 0.0, np.exp(arg) / hs[:, 1:]) * (error(arg) + 2)
    for row in range(tokens):
        np.add.at(err[row], hi[row][ok[row]], (q_off + 3 * q)[row][ok[row]])
    assert (np.abs(host(dz) - back) <= U * err + (U + HALF[dtype]) * np.abs(back) + TINY).all()

    # two shards, the first without row 1's largest logits' second
    cut = 300
    parts = torch.empty(2, tokens, 4, device="cuda")
    ops.distill_shard(z[:, :cut], ids, t, parts[0], first=0, vocab=vocab, temperature=tau)
    ops.distill_shard(z[:, cut:], ids, t, parts[1], first=cut, vocab=vocab, temperature=tau)
    loss2, stats2, dz2 = torch.empty_like(loss), torch.empty_like(stats), torch.empty(tokens, vocab - cut, dtype=z.dtype, device="cuda")
    ops.distill_join(parts, ids, t, loss2, stats2, vocab=vocab, temperature=tau)
    assert torch.equal(stats2[:, 0], stats[:, 0])
    assert (np.abs(host(stats2[:, 1]) - s) <= s_off + U * s).all()
    at = np.where(ok, hi, 0)
    sizes = np.zeros(tokens)
    for a, b in ((0, cut), (cut, vocab)):
        here = ok & (hi >= a) & (hi < b)
        ms = hz[:, a:b].max(axis=1)
        gap = np.where(here & (q > 0), np.abs(np.take_along_axis(hz, at, axis=1) - ms[:, None]) / tau32, 0.0)
        sizes += (q * gap).sum(axis=1) + (q * here).sum(axis=1) * np.abs(ms - m) / tau32
    assert (np.abs(host(loss2) - want) <= off + U * (sizes + 2)).all(), (host(loss2), want)
    ops.distill_backward(z[:, cut:], ids, t, stats, dz2, temperature=tau, scale=tau, first=cut, vocab=vocab)
    assert torch.equal(dz2, dz[:, cut:])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("up,tau", [(2.0 ** 100, 2.0 ** -40), (-2.0 ** 127, 2.0 ** -10), (2.0 ** 120, 2.0 ** -64)])
def test_factors_beyond_binary32(torch, ops, up, tau, dtype):
    """dloss * scale / temperature is, the gradient of shares far below 1 is not: masked columns have gradient 0, and one
    whose share and choice are nearly the same has their difference."""
    tokens, vocab = 12, 600
    g = np.random.default_rng(3)
    # distances from the top in units of the temperature, exact in both types
    z = -(40 + np.floor(g.uniform(0, 60, (tokens, vocab)))) * tau
    z[:, 7], z[:, 11], z[:, 599] = 0.0, -np.inf, -np.inf
    ids = np.tile(np.array([[7, 20, 300]]), (tokens, 1))
    t = np.tile(np.array([[0.0, -45.0, -64.0]]) * tau, (tokens, 1))
    ids[3] = -1
    logits = torch.from_numpy(z.astype(np.float32)).to(getattr(torch, dtype)).cuda()
    teacher = torch.from_numpy(t.astype(np.float32)).cuda()
    hi = torch.from_numpy(ids).cuda()
    loss, stats, dz = torch.empty(tokens, device="cuda"), torch.empty(tokens, 2, device="cuda"), torch.empty_like(logits)
    ops.distill(logits, hi, teacher, loss, stats, temperature=tau)
    dloss = torch.full((tokens,), up, device="cuda")
    ops.distill_backward(logits, hi, teacher, stats, dz, dloss=dloss, scale=0.75, temperature=tau)
    got, hz, hs = host(dz), host(logits), host(stats)
    want = ref.distill_backward(hz, ids, host(teacher), tau, hs, np.full(tokens, up * 0.75))
    assert (got[:, [11, 599]] == 0).all() and (got[3] == 0).all() and not np.isnan(got).any()
    with np.errstate(all="ignore"):
        arg = np.where(np.isinf(hz), 0.0, (hz - hs[:, :1]) / tau)
        err = np.where(np.isinf(hz), 0.0, np.exp(arg) / hs[:, 1:]) * (error(arg) + 4)
    q, logq, ok = ref.choices(ids, host(teacher), vocab, tau)
    r = error(np.where(q > 0, logq, 0.0))
    for row in range(tokens):
        np.add.at(err[row], ids[row][ok[row]], (q * (r + (q * r).sum(axis=1, keepdims=True) + 5))[row][ok[row]])
    # exp(-88) is below 2^-126 and taken as 0 (the head of this file): off by the whole of such a share, p < 2^-126,
    # times the factor, 2^-126 * 2^139.6 = 1.2e4 where the other terms are 0.1
    err = (U * err + 2.0 ** -126) * abs(up) * 0.75 / tau + (U + HALF[dtype]) * np.abs(want)
    largest = float(torch.finfo(getattr(torch, dtype)).max)
    inside = np.abs(want) + err < largest
    assert inside[:, 20:].any()
    assert (np.abs(got - want)[inside] <= err[inside]).all()
    over = np.abs(want) - err > largest
    assert np.isinf(got[over]).all() and (np.sign(got[over]) == np.sign(want[over])).all()


def test_small_shares_with_a_large_factor(torch, ops):
    """Shares of 2^-120 to 2^-142, whose exponentials are normal numbers, and a factor of 2^140: each gradient to its
    relative bound."""
    vocab, n = 131072, 16
    z = torch.zeros(3, vocab, device="cuda")
    z[:, :n] = -torch.arange(72.0, 72.0 + n, device="cuda")
    ids, t = torch.full((3, 1), vocab - 1, device="cuda"), torch.zeros(3, 1, device="cuda")
    loss, stats, dz = torch.empty(3, device="cuda"), torch.empty(3, 2, device="cuda"), torch.empty_like(z)
    ops.distill(z, ids, t, loss, stats)
    ops.distill_backward(z, ids, t, stats, dz, dloss=torch.full((3,), 2.0 ** 100, device="cuda"), scale=2.0 ** 40)
    hz, hs = host(z)[:, :n], host(stats)
    want = np.exp(hz - hs[:, :1]) / hs[:, 1:] * 2.0 ** 140
    assert (np.abs(host(dz)[:, :n] - want) <= U * (error(hz) + 4) * want).all()
