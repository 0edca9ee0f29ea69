"""The routing gradient in every shape that it is compiled for: numbers of
experts around each bound, rows of whole 16-byte units and others, one choice
a lane and two (topk above 16 where 16 lanes share a token); and the last part
of a call that is split into launches.

Bounds (u = 2^-24), as in tests/test_gpu_ops_route.py: 128 u of the terms'
magnitudes (score * (|a| + sum |r a|)) and half a step of the type."""
from __future__ import annotations

import numpy as np
import pytest

import ops_reference as ref
from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24
DT = {"f32": "float32", "bf16": "bfloat16"}


def ops():
    from copy_reduce_snac_amd import operators

    return operators


SHAPES = [(n, k) for n in (1, 3, 16, 17, 63, 65, 100, 120, 127, 128, 130, 255, 257, 264, 300, 504, 511, 512, 520, 1000)
          for k in (1, 7, 17, 32) if k <= n]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("n,topk", SHAPES)
def test_shapes(dtype, score, renorm, n, topk):
    import torch

    g = np.random.default_rng(n * 40 + topk)
    tokens = 13
    x = torch.tensor((g.normal(size=(tokens, n)) * 2).astype(np.float32), device="cuda")
    x[2, ::3] = -np.inf
    x[3] = -np.inf
    x[4] -= 80.0
    x = x.to(getattr(torch, DT[dtype]))
    xs = x.double().cpu().numpy()
    ids = np.stack([g.permutation(n)[:topk] for _ in range(tokens)]).astype(np.int32)
    ids[2] = [i if i % 3 else -1 for i in ids[2]]
    ids[3] = -1
    ids[5, topk // 2] = n + 5
    ids[6, -1] = -7
    dw = g.normal(size=(tokens, topk)).astype(np.float32)
    dx = torch.full((tokens + 1, n), 77.0, dtype=x.dtype, device="cuda")
    ops().route_backward(x, torch.tensor(ids, device="cuda"), torch.tensor(dw, device="cuda"), dx[:-1], score=score,
                         renorm=renorm, scale=2.5)
    assert bool((dx[-1] == 77).all())
    got = dx[:-1].double().cpu().numpy()
    for t in range(tokens):
        want = ref.route_backward(xs[t], ids[t], dw[t], score, renorm, 2.5)
        have = [(int(i), 2.5 * abs(float(d))) for i, d in zip(ids[t], dw[t]) if 0 <= i < n]
        size = np.zeros(n)
        if have:
            at, a = np.array([i for i, _ in have]), np.array([d for _, d in have])
            s = ref.scores(xs[t], score)
            r = ref.chosen_scores(xs[t], s, at, score, renorm)
            if score == "softmax" and not renorm:
                size[at] = a
                size = s * (size + np.dot(r, a))
            else:
                size[at] = r * (a + (np.dot(r, a) if renorm else 0))
        tol = 128 * U * size + ref.half_step(dtype) * np.abs(want) * 1.01 + 1e-37
        assert np.all(np.abs(got[t] - want) <= tol), (t, np.max(np.abs(got[t] - want) - tol))


def test_last_part_of_a_split_call():
    """2^28 tokens and some are more than two launches: the tokens of the last one have the gradient that they have
    in a call of their own, and the weights of their logits."""
    import torch

    n, last = 2 ** 28 + 77, 500
    x = torch.empty(n, 16, dtype=torch.bfloat16, device="cuda").normal_()
    w, ids = torch.empty(n, 2, device="cuda"), torch.empty(n, 2, dtype=torch.int32, device="cuda")
    dw = torch.empty(n, 2, device="cuda").normal_()
    dx = torch.empty_like(x)
    ops().route(x, w, ids, renorm=False)
    ops().route_backward(x, ids, dw, dx, renorm=False)
    own = torch.empty_like(dx[-last:])
    ops().route_backward(x[-last:], ids[-last:], dw[-last:], own, renorm=False)
    assert torch.equal(dx[-last:], own)
    xs, dws = x[-last:].double().cpu().numpy(), dw[-last:].cpu().numpy()
    got_w, got_ids = w[-last:].double().cpu().numpy(), ids[-last:].cpu().numpy()
    for t in range(0, last, 7):
        rw, rid = ref.route(xs[t], 2, renorm=False)
        assert got_ids[t].tolist() == rid.tolist() and np.all(np.abs(got_w[t] - rw) <= 96 * U * rw), t
        want = ref.route_backward(xs[t], rid, dws[t], "softmax", False, 1.0)
        size = ref.scores(xs[t], "softmax") * (np.abs(dws[t]).sum() * 2)
        tol = 128 * U * size + ref.half_step("bf16") * np.abs(want) * 1.01
        assert np.all(np.abs(own[t].double().cpu().numpy() - want) <= tol), t
