"""examples/distill_step.py: layer norm, routing with its balance loss, the
experts and the distillation over shards of the vocabulary, with the
collectives between them, against the same model in binary64 with torch's
autograd and the experts that the routing chose.  The example rounds each
activation and its gradient to bf16: about twelve roundings of half a step,
2^-8, on the longest path to a gradient (embedding, norm, expert, combine, sum,
norm, logits; the gradients of logits, rows, norm, combine, expert, norm, sum),
in the 2-norm below their sum, 14 * 2^-8 = 5.5e-2; the loss's own below that."""
from __future__ import annotations

import os
import sys

import pytest

from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUND = 14 * 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import distill_step
    finally:
        sys.path.pop(0)
    return distill_step


def norm(torch, x, w, b):
    d = x - x.mean(dim=1, keepdim=True)
    return d / torch.sqrt((d * d).mean(dim=1, keepdim=True) + 1e-5) * w + b


def test_gradients_against_autograd(example):
    import torch

    torch.cuda.set_device(0)
    m = example.DistillStep(ranks=4, tokens=70, width=64, vocab=512, experts=6, topk=2, choices=9)
    try:
        loss, ids = m.forward_backward()
        torch.cuda.synchronize()
        table = torch.cat(m.tables).double().cpu().requires_grad_()
        router = m.router.double().cpu().requires_grad_()
        matrices = m.matrices.double().cpu().requires_grad_()
        norms = torch.stack(m.norms).double().cpu().requires_grad_()
        at = torch.cat(ids).long().cpu()
        assert int(at.min()) >= 0
        x = table[torch.cat(m.ids).cpu()] * m.width ** 0.5
        h = norm(torch, x, norms[0], norms[1])
        p = torch.softmax(h @ router, dim=1)
        w = p.gather(1, at)
        w = w / w.sum(dim=1, keepdim=True)
        mixed = sum(w[:, k:k + 1] * (h.unsqueeze(1) @ matrices[at[:, k]]).squeeze(1) for k in range(m.topk))
        counts = torch.bincount(at.flatten(), minlength=m.experts).double()
        balance = m.balance * m.experts * (counts / counts.sum() * p.mean(dim=0)).sum()
        y = norm(torch, x + mixed, norms[2], norms[3])
        logp = torch.log_softmax(y @ table.t() / m.temperature, dim=1)
        chosen, teacher = m.chosen.cpu(), m.teacher.double().cpu()
        some = (chosen >= 0).all(dim=1)
        logq = torch.log_softmax(teacher[some] / m.temperature, dim=1)
        kl = (logq.exp() * (logq - logp[some].gather(1, chosen[some]))).sum()
        want = kl * m.temperature ** 2 / (m.n * m.tokens) + balance
        want.backward()

        def off(got, exact):
            return float((got.double().cpu() - exact).norm() / exact.norm())

        assert abs(float(loss) - want.item()) <= BOUND * want.item()
        assert off(torch.cat(m.dtables), table.grad) <= BOUND
        assert off(m.drouter[0], router.grad) <= BOUND
        assert off(m.dmatrices[0], matrices.grad) <= BOUND
        for i in range(4):
            assert off(m.dnorms[0][i], norms.grad[i]) <= BOUND, i
        for grads in (m.drouter, m.dmatrices, m.dnorms):
            assert all(torch.equal(d, grads[0]) for d in grads)
    finally:
        m.close()


def test_steps(example):
    import math

    losses = example.main(["--steps", "3", "--tokens", "64", "--width", "128", "--vocab", "1024"])
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
