"""Softmax statistics of a confident router on the GPU: one logit far above
many, whose scores are each below half a step of the sum.

Bounds (u = 2^-24).  The low scores are exponentials of an exact difference d =
-17: the product with log2(e) and that constant are off by 17 (1 + 0.23) u, the
exponential by 2 u: 23 u.  All of them together are 1e-5 of the sum, so the sum
is off by 23e-5 u, and the top's weight by that and one rounding.  1 - weight is
off by 23 u, and the top's gradient, weight * a * (1 - weight), by one
rounding more and the estimate of the reciprocal (2^-40, over 1e-5 below u):
26 u.  With bf16 logits that is a product of three binary32 numbers (30 u) and
half a step."""
from __future__ import annotations

import numpy as np
import pytest

from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24


@pytest.mark.parametrize("tokens", [5, 4100])
@pytest.mark.parametrize("experts", [60, 128, 256, 500, 1024])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("biased", [False, True])
def test_confident_router(tokens, experts, dtype, biased):
    import torch

    from copy_reduce_snac_amd import operators as ops

    x = torch.full((tokens, experts), -17.0, device="cuda", dtype=getattr(torch, dtype))
    top = torch.arange(tokens, device="cuda") * 7 % experts
    x[torch.arange(tokens, device="cuda"), top] = 0.0
    bias = torch.zeros(experts, device="cuda") if biased else None
    w, ids = torch.empty(tokens, 2, device="cuda"), torch.empty(tokens, 2, dtype=torch.int32, device="cuda")
    ops.route(x, w, ids, bias=bias, renorm=False)
    assert torch.equal(ids[:, 0], top.int())
    low = np.exp(-17.0)
    total = 1.0 + (experts - 1) * low
    assert float((w[:, 0].double() * total - 1.0).abs().max()) <= 1.01 * U
    # one choice, the top: the gradient of its weight
    dx = torch.empty_like(x)
    dw = torch.rand(tokens, 1, device="cuda") + 0.5
    ops.route_backward(x, ids[:, :1].contiguous(), dw, dx, renorm=False)
    s = 1.0 / total
    tol = 26 * U if dtype == "float32" else 30 * U + 2.0 ** -8
    a = dw[:, 0].double()
    got = dx.double().gather(1, top[:, None])[:, 0]
    want = a * s * ((experts - 1) * low / total)
    assert float((got / want - 1.0).abs().max()) <= tol
    # and of the others, which it takes away from: weight and score as above, and one rounding
    rest = dx.double().scatter(1, top[:, None], 0.0).sum(1)
    assert float((rest / -want - 1.0).abs().max()) <= tol


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_nearly_one_choice(score):
    """Renormalised weights of two choices, one of them 1 - 1e-7: its gradient is what is left of 1, in relative terms
    (r = 1 / (1 + q) for the ratio q of the scores, off by two exponentials of 17 and 3 of at most 2 u and 17 u)."""
    import torch

    from copy_reduce_snac_amd import operators as ops

    x = torch.full((300, 64), -3.0, device="cuda")
    x[:, 5], x[:, 40] = (0.0, -16.0) if score == "softmax" else (-1.0, -17.0)
    ids = torch.tensor([[5, 40]] * 300, dtype=torch.int32, device="cuda")
    dw = torch.rand(300, 2, device="cuda") + torch.tensor([1.0, 3.0], device="cuda")
    dx = torch.empty_like(x)
    ops.route_backward(x, ids, dw, dx, score=score, renorm=True)
    a = dw.double()
    sc = lambda v: np.exp(v) if score == "softmax" else 1 / (1 + np.exp(-v))  # noqa: E731
    x0, x1 = float(x[0, 5]), float(x[0, 40])
    q = sc(x1) / sc(x0)
    r0, r1 = 1 / (1 + q), q / (1 + q)
    far = (1.0, 1.0) if score == "softmax" else (sc(-x0), sc(-x1))
    d = a[:, 0] - a[:, 1]
    for at, want in ((5, r0 * r1 * far[0] * d), (40, -r0 * r1 * far[1] * d)):
        got = dx[:, at].double()
        assert float((got / want - 1.0).abs().max()) <= 48 * U, at
    assert not bool(dx[:, :5].any()) and not bool(dx[:, 41:].any())
