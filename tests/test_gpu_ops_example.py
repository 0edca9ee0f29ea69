"""examples/moe_step.py: the operators and the collectives together, against
the same layer in binary64 with torch's autograd and the experts that the
routing chose.  The example rounds each activation and its gradient to bf16
(about eight roundings of half a step, 2^-8, on the longest path to a table's
gradient, in the 2-norm below their sum, 8 * 2^-8 = 3.1e-2)."""
from __future__ import annotations

import os
import sys

import pytest

from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUND = 8 * 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import moe_step
    finally:
        sys.path.pop(0)
    return moe_step


def test_gradients_against_autograd(example):
    import torch

    torch.cuda.set_device(0)
    m = example.MoeStep(ranks=4, tokens=96, width=64, vocab=512, experts=16, topk=3)
    try:
        loss, ids = m.forward_backward()
        torch.cuda.synchronize()
        table = torch.cat(m.tables).double().cpu().requires_grad_()
        router = m.router.double().cpu().requires_grad_()
        weights = torch.cat(m.weights).double().cpu().requires_grad_()
        x = table[torch.cat(m.ids).cpu()] * m.width ** 0.5
        s = torch.sigmoid(x @ router)
        at = torch.cat(ids).long().cpu()
        assert int(at.min()) >= 0
        w = s.gather(1, at)
        w = 2.5 * w / w.sum(dim=1, keepdim=True)
        out = sum(w[:, k:k + 1] * (x.unsqueeze(1) @ weights[at[:, k]]).squeeze(1) for k in range(m.topk))
        want = ((out - torch.cat(m.target).double().cpu()) ** 2).sum() / (2 * m.n * m.tokens)
        want.backward()

        def off(got, exact):
            return float((got.double().cpu() - exact).norm() / exact.norm())

        assert abs(float(loss) - want.item()) <= BOUND * want.item()
        assert off(torch.cat(m.dtables), table.grad) <= BOUND
        assert off(torch.cat(m.dweights), weights.grad) <= BOUND
        assert off(m.drouter[0], router.grad) <= BOUND
        assert all(torch.equal(d, m.drouter[0]) for d in m.drouter)
    finally:
        m.close()


def test_steps(example):
    losses = example.main(["--steps", "4", "--tokens", "128", "--width", "128"])
    assert len(losses) == 4 and losses[-1] < losses[0]
