"""The loss against a teacher's top logits and its gradient on the GPU, against
tests/ops_step_reference.py.

Bounds, u = 2^-24.  An exponential of (x - top) / temperature is off by
(2 + 2.5 |arg|) u of itself (subtraction, product with a rounded factor, the
hardware's exponential).
  S     the terms' errors, and 8 u of the sum (7 additions of a unit, a rounding)
  q     q (r + sum q r + 2) u with r = 2 + 2.5 |arg|
  loss  sum of q's errors times |log q - log p|, S's and the teacher's sum's
        relative errors, a rounding; joined from shards also the roundings of
        each part: D, S and Q
  dz    for the stats that the call got: |factor| u (p (r + 4) + q's error + 2 q)
        and half a step
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


def teacher_errors(ids, t, vocab, tau):
    """q, log q, validity, q's error and the relative error of the teacher's sum, in units of u."""
    q, logq, ok = ref.choices(ids, t, vocab, tau)
    arg = np.where(ok, logq - np.where(ok, logq, -np.inf).max(axis=1, keepdims=True, initial=-1e30), 0.0)
    r = 2 + 2.5 * np.abs(arg)
    rel = (q * r).sum(axis=1, keepdims=True)
    return q, logq, ok, q * (r + rel + 2), rel


def row_errors(z, tau):
    """The largest logit, S and S's relative error in units of u; the exponent's distances."""
    m = z.max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        arg = np.where(z == -np.inf, 0.0, (z - np.where(np.isinf(m), 0, m)) / tau)
        e = np.where(z == -np.inf, 0.0, np.exp(arg))
    s = e.sum(axis=1, keepdims=True)
    r = 2 + 2.5 * np.abs(arg)
    return m, s, np.where(s > 0, (e * r).sum(axis=1, keepdims=True) / np.where(s > 0, s, 1) + 8, 0.0), r


def loss_bound(z, ids, t, tau, loss):
    q, logq, ok, q_off, rel = teacher_errors(ids, t, z.shape[1], tau)
    m, s, s_rel, _ = row_errors(z, tau)
    with np.errstate(all="ignore"):
        logp = np.take_along_axis((z - m) / tau - np.log(s), np.where(ok, ids, 0), axis=1)
        gap = np.where(q > 0, np.abs(logq - logp), 0.0)
    return U * ((q_off * (gap + 1)).sum(axis=1) + s_rel[:, 0] + rel[:, 0] + np.abs(loss)) + TINY


def inputs(torch, tokens, vocab, topk, dtype, tdtype, itype, seed, shift=0, spread=1.0):
    g = np.random.default_rng(seed)
    z = spread * g.normal(size=(tokens, vocab))
    t = 2.0 + 2 * g.normal(size=(tokens, topk))
    ids = np.argsort(g.random((tokens, vocab)), axis=1)[:, :topk] if vocab < 4000 else g.integers(0, vocab, (tokens, topk))
    ids = np.resize(ids, (tokens, topk)).astype(np.int64)
    for r in range(tokens):
        z[r, ids[r]] = t[r] + 0.5 * g.normal(size=topk)
    if vocab > 8:
        z[:, 5] = np.where((ids == 5).any(axis=1), z[:, 5], -np.inf)  # a masked column that nobody chose
    if tokens > 6:
        ids[1] = -1                                   # no choice
        ids[2, 0], ids[3, 0] = vocab, -(2 ** 31)      # no columns
        t[4, 0] = -np.inf                             # a masked choice
        t[5] = -np.inf                                # all of them masked
        ids[6] = ids[6, 0]                            # one column in all choices
    wide = torch.full((tokens + 1, shift + vocab + 3), 77.0, dtype=getattr(torch, DT[dtype]), device="cuda")
    logits = wide[:tokens, shift:shift + vocab]
    logits.copy_(torch.from_numpy(z.astype(np.float32)))
    return (wide, logits, torch.from_numpy(ids).to(getattr(torch, itype)).cuda(),
            torch.from_numpy(t.astype(np.float32)).to(getattr(torch, DT[tdtype])).cuda())


SHAPES = [(1, 1, 1, 1.0), (9, 2, 1, 1.0), (8, 11, 3, 0.5), (33, 64, 4, 2.0), (7, 255, 70, 1.0), (17, 1000, 8, 1.5), (8, 2048, 256, 3.0),
          (9, 2049, 64, 1.0), (8, 4096, 65, 1.0), (12, 8195, 20, 1.0), (9, 32768, 130, 2.0), (8, 50001, 64, 1.0), (700, 9001, 5, 1.0)]


@pytest.mark.parametrize("dtype,tdtype,itype", [("f32", "f32", "int64"), ("bf16", "bf16", "int64"), ("bf16", "f32", "int32"),
                                                ("f32", "bf16", "int32")])
@pytest.mark.parametrize("tokens,vocab,topk,tau", SHAPES)
def test_both_ways(torch, ops, dtype, tdtype, itype, tokens, vocab, topk, tau):
    shift = vocab % 4
    wide, logits, ids, t = inputs(torch, tokens, vocab, topk, dtype, tdtype, itype, vocab + topk, shift)
    loss = torch.full((tokens + 1,), 55.0, device="cuda")
    stats = torch.full((tokens + 1, 2), 55.0, device="cuda")
    ops.distill(logits, ids, t, loss[:tokens], stats[:tokens], temperature=tau)
    torch.cuda.synchronize()
    assert loss[-1] == 55 and (stats[-1] == 55).all()
    hz, hi, ht = host(logits), ids.cpu().numpy().astype(np.int64), host(t)
    want, m, s = ref.distill(hz, hi, ht, tau)
    _, _, s_rel, r = row_errors(hz, tau)
    assert np.array_equal(host(stats[:tokens, 0]), m)
    assert (np.abs(host(stats[:tokens, 1]) - s) <= U * (s_rel[:, 0] + 1) * s).all()
    assert (np.abs(host(loss[:tokens]) - want) <= loss_bound(hz, hi, ht, tau, want)).all()

    up = torch.rand(tokens, device="cuda") + 0.5
    dz = torch.full((tokens + 1, vocab + 5), 77.0, dtype=logits.dtype, device="cuda")
    ops.distill_backward(logits, ids, t, stats[:tokens], dz[:tokens, 2:2 + vocab], dloss=up, scale=0.375, temperature=tau)
    torch.cuda.synchronize()
    assert (dz[tokens:] == 77).all() and (dz[:, :2] == 77).all() and (dz[:, 2 + vocab:] == 77).all() and (wide[tokens:] == 77).all()
    hs = host(stats[:tokens])
    want = ref.distill_backward(hz, hi, ht, tau, hs, host(up) * 0.375)
    q, _, ok, q_off, _ = teacher_errors(hi, ht, vocab, tau)
    with np.errstate(all="ignore"):
        err = np.where(np.isinf(hz), 0.0, np.exp((hz - hs[:, :1]) / tau) / hs[:, 1:]) * (r + 4)
    for row in range(tokens):
        np.add.at(err[row], hi[row][ok[row]], (q_off + 3 * q)[row][ok[row]])
    err = err * U * (host(up) * 0.375 / tau)[:, None] + (U + HALF[dtype]) * np.abs(want) + TINY
    got = host(dz[:tokens, 2:2 + vocab])
    assert (np.abs(got - want) <= err).all(), np.abs(got - want).max()
    assert (got[~ok.any(axis=1)] == 0).all()
    # in place, and all factors 1
    same = logits.clone()
    ops.distill_backward(same, ids, t, stats[:tokens], same, dloss=up, scale=0.375, temperature=tau)
    assert torch.equal(same, dz[:tokens, 2:2 + vocab])
    a, b = torch.empty_like(same), torch.empty_like(same)
    ops.distill_backward(logits, ids, t, stats[:tokens], a, temperature=tau)
    ops.distill_backward(logits, ids, t, stats[:tokens], b, dloss=torch.ones(tokens, device="cuda"), temperature=tau)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cuts", [[0, 3000], [0, 1000, 3000], [0, 1, 1, 1500, 2999, 3000], list(range(0, 3001, 200)) + [3000]])
def test_shards(torch, ops, dtype, cuts):
    tokens, vocab, topk, tau = 40, 3000, 24, 1.25
    _, logits, ids, t = inputs(torch, tokens, vocab, topk, dtype, "f32", "int64", 3)
    n = len(cuts) - 1
    parts = torch.full((n, tokens, 4), 55.0, device="cuda")
    spans = [slice(a, b) for a, b in zip(cuts, cuts[1:])]
    order = list(range(n))[::-1]
    for slot, i in enumerate(order):  # in any order
        ops.distill_shard(logits[:, spans[i]], ids, t, parts[slot], first=cuts[i], vocab=vocab, temperature=tau)
    loss, stats = torch.empty(tokens, device="cuda"), torch.empty(tokens, 2, device="cuda")
    ops.distill_join(parts, ids, t, loss, stats, vocab=vocab, temperature=tau)
    hz, hi, ht = host(logits), ids.cpu().numpy().astype(np.int64), host(t)
    want, m, s = ref.distill(hz, hi, ht, tau)
    _, _, s_rel, _ = row_errors(hz, tau)
    assert np.array_equal(host(stats[:, 0]), m)
    # a part's S is rounded once more, and the joint one
    assert (np.abs(host(stats[:, 1]) - s) <= U * (s_rel[:, 0] + 2) * s).all()
    # D is a mean of |z - m| / tau over the choices, Q at most 1
    sizes = np.zeros(tokens)
    q, _, ok = ref.choices(hi, ht, vocab, tau)
    at = np.where(ok, hi, 0)
    for sp in spans:
        if sp.stop == sp.start:
            continue
        here = ok & (hi >= sp.start) & (hi < sp.stop)
        ms = hz[:, sp].max(axis=1)
        ms = np.where(np.isinf(ms), 0.0, ms)
        gap = np.where(here, np.abs(np.take_along_axis(hz, at, axis=1) - ms[:, None]) / tau, 0.0)
        sizes += (q * gap).sum(axis=1) + (q * here).sum(axis=1) * np.abs(ms - m) / tau
    assert (np.abs(host(loss) - want) <= loss_bound(hz, hi, ht, tau, want) + U * (sizes + 2)).all()
    # the shards' gradients are the whole row's
    whole = torch.empty_like(logits)
    ops.distill_backward(logits, ids, t, stats, whole, scale=0.5, temperature=tau)
    for i, sp in enumerate(spans):
        z = logits[:, sp].contiguous()
        dz = torch.empty_like(z)
        ops.distill_backward(z, ids, t, stats, dz, scale=0.5, first=cuts[i], vocab=vocab, temperature=tau)
        assert torch.equal(dz, whole[:, sp]), i


def test_shards_without_logits(torch, ops):
    """A shard that only pads the vocabulary: its columns are masked, and have no part."""
    tokens, vocab, topk = 20, 300, 6
    _, logits, ids, t = inputs(torch, tokens, vocab, topk, "f32", "f32", "int32", 9)
    z = torch.cat([logits, torch.full((tokens, 50), -float("inf"), device="cuda")], dim=1)
    ids = torch.where(ids == vocab, torch.full_like(ids, -1), ids)  # vocab is a column now
    loss, stats = torch.empty(tokens, device="cuda"), torch.empty(tokens, 2, device="cuda")
    ops.distill(logits, ids, t, loss, stats)
    parts = torch.empty(2, tokens, 4, device="cuda")
    ops.distill_shard(z[:, :vocab], ids, t, parts[0], first=0, vocab=350)
    ops.distill_shard(z[:, vocab:], ids, t, parts[1], first=vocab, vocab=350)
    assert bool((parts[1, :, 0] == -float("inf")).all()) and bool((parts[1, :, 1:] == 0).all())
    loss2, stats2 = torch.empty(tokens, device="cuda"), torch.empty(tokens, 2, device="cuda")
    ops.distill_join(parts, ids, t, loss2, stats2, vocab=350)
    assert torch.equal(stats, stats2)
    assert float((loss - loss2).abs().max()) <= 2 * U * float(loss.max() + parts[0, :, 2].abs().max() + 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masks(torch, ops, dtype):
    """Rows and choices that are masked; the type's lowest value is no mask."""
    inf, low = float("inf"), torch.finfo(getattr(torch, DT[dtype])).min
    z = torch.randn(8, 40, device="cuda")
    z[0] = -inf                   # all masked: no part
    z[1] = low                    # all the lowest: even
    z[2, :39] = low               # all but one
    z[3, 7] = -inf                # a choice of a masked column
    z[4] = 1e30
    z[5, 3] = inf
    z[6, 3] = float("nan")
    z = z.to(getattr(torch, DT[dtype]))
    ids = torch.tensor([[7, 39]] * 8, dtype=torch.int32, device="cuda")
    t = torch.zeros(8, 2, device="cuda")
    t[7, 0] = float("nan")
    loss, stats, dz = torch.empty(8, device="cuda"), torch.empty(8, 2, device="cuda"), torch.empty_like(z)
    ops.distill(z, ids, t, loss, stats)
    ops.distill_backward(z, ids, t, stats, dz)
    v = loss.tolist()
    assert v[0] == 0 and bool((dz[0] == 0).all())
    even = np.log(40) - np.log(2)
    assert abs(v[1] - even) <= 16 * U * even and abs(v[4] - even) <= 16 * U * even
    want = np.full(40, 1 / 40)
    want[[7, 39]] -= 0.5
    assert (np.abs(host(dz[1]) - want) <= (16 * U + HALF[dtype]) * np.abs(want)).all()
    assert v[2] > 1e37 or v[2] == inf
    assert dz[2, 39] == 0.5 and dz[2, 7] == -0.5 and float(dz[2].float().abs().sum()) == 1.0
    assert v[3] == inf and dz[3, 7] == -0.5 and not dz[3].isnan().any()
    for r in (5, 6, 7):
        assert np.isnan(v[r]), r
    assert bool(dz[5].isnan().all()) and bool(dz[6].isnan().all())
    assert dz[7].isnan().nonzero().flatten().tolist() == [7, 39]
    dloss = torch.ones(8, device="cuda")
    dloss[0], dloss[1] = float("nan"), float("nan")
    ops.distill_backward(z, ids, t, stats, dz, dloss=dloss)
    assert bool((dz[0] == 0).all()) and bool(dz[1].isnan().all())


@pytest.mark.parametrize("tau", [2.0 ** -64, 1e-4, 30.0, 2.0 ** 64])
def test_temperatures(torch, ops, tau):
    _, logits, ids, t = inputs(torch, 12, 500, 9, "f32", "f32", "int64", 21)
    loss, stats, dz = torch.empty(12, device="cuda"), torch.empty(12, 2, device="cuda"), torch.empty(12, 500, device="cuda")
    ops.distill(logits, ids, t, loss, stats, temperature=tau)
    ops.distill_backward(logits, ids, t, stats, dz, temperature=tau, scale=tau)
    hz, hi, ht = host(logits), ids.cpu().numpy(), host(t)
    tau = float(np.float32(tau))
    want, m, s = ref.distill(hz, hi, ht, tau)
    assert not loss.isnan().any() and not dz.isnan().any()
    if tau > 1:  # where it is tiny the largest logit is all that counts
        assert (np.abs(host(loss) - want) <= loss_bound(hz, hi, ht, tau, want)).all()
        back = ref.distill_backward(hz, hi, ht, tau, host(stats), np.full(12, tau))
        assert (np.abs(host(dz) - back) <= 32 * U).all()
    else:
        assert (host(stats)[:, 1] >= 1).all()


def test_small_losses(torch, ops):
    """A student that is nearly the teacher: the loss is a small difference of large sums."""
    tokens, vocab = 64, 4001
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    z = torch.full((tokens, vocab), -40.0, device="cuda")
    ids = torch.arange(32, device="cuda").repeat(tokens, 1) * 100 + 3
    t = torch.randn(tokens, 32, generator=g, device="cuda") * 2
    z.scatter_(1, ids, t + 0.01 * torch.randn(tokens, 32, generator=g, device="cuda"))
    loss, stats = torch.empty(tokens, device="cuda"), torch.empty(tokens, 2, device="cuda")
    ops.distill(z, ids, t, loss, stats)
    want, _, _ = ref.distill(host(z), ids.cpu().numpy(), host(t), 1.0)
    assert want.max() < 2e-4
    assert (np.abs(host(loss) - want) <= loss_bound(host(z), ids.cpu().numpy(), host(t), 1.0, want)).all()


def test_long_offsets(torch, ops):
    """Rows whose elements lie past 2^32 bytes from the first."""
    tokens, vocab = 17000, 131072  # 4.46 GB of bf16
    z = torch.zeros(tokens, vocab, dtype=torch.bfloat16, device="cuda")
    ids = (torch.arange(tokens, device="cuda").unsqueeze(1) * 7 + torch.arange(2, device="cuda")).to(torch.int32) % vocab
    z.scatter_(1, ids.long(), 4.0)
    t = torch.zeros(tokens, 2, device="cuda")
    loss, stats = torch.empty(tokens, device="cuda"), torch.empty(tokens, 2, device="cuda")
    ops.distill(z, ids, t, loss, stats)
    s = 2 + (vocab - 2) * np.exp(-4.0)
    assert bool((stats[:, 0] == 4).all()) and float((stats[:, 1] - s).abs().max()) <= 24 * U * s
    want = np.log(0.5) + np.log(s)
    assert float((loss - want).abs().max()) <= 32 * U * want
    ops.distill_backward(z, ids, t, stats, z)
    p = 1 / s
    assert float((z.gather(1, ids.long()).double() - (p - 0.5)).abs().max()) <= 0.5 * 2.0 ** -8
    assert float((z[-1].double().sum() - z[-1].gather(0, ids[-1].long()).double().sum()) / (p * np.exp(-4.0) * (vocab - 2)) - 1) <= 2.0 ** -8


def test_no_tokens(torch, ops):
    z, ids, t = torch.empty(0, 9, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    loss, stats = torch.empty(0, device="cuda"), torch.empty(0, 2, device="cuda")
    ops.distill(z, ids, t, loss, stats)
    ops.distill_join(torch.empty(3, 0, 4, device="cuda"), ids, t, loss, stats, vocab=9)
    ops.distill_backward(z, ids, t, stats, z)
    # a shard of no columns has no part either
    ids, t, part = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, device="cuda"), torch.ones(3, 4, device="cuda")
    empty = torch.empty(3, 0, device="cuda")
    ops.distill_shard(empty, ids, t, part, first=9, vocab=9)
    assert part.tolist() == [[-float("inf"), 0, 0, 0]] * 3
    ops.distill_backward(empty, ids, t, torch.ones(3, 2, device="cuda"), empty, first=9, vocab=9)
