"""Training steps of a small mixture-of-experts language model against a
teacher's top logits, over N logical ranks: the operators of
``copy_reduce_snac_amd.operators`` around the collectives of
``copy_reduce_snac_amd.tensors``.

Rank r holds a shard of the vocabulary and tokens of its own; the experts, the
router and the norms are on every rank, their gradients are summed.  One step:

  embedding        every shard looks up all ranks' tokens; reduce_scatter sums
                   the shards and leaves each rank its tokens' rows x
  experts          h = layer_norm(x); route, dispatch, a matrix an expert
                   (torch), combine: m; all_reduce of the ranks' loads and the
                   balance loss
  logits           y = layer_norm(x + m); all_gather; each rank's columns of
                   the logits are y times its shard of the table
  distillation     distill_shard, all_gather of the parts, distill_join
  backward         the same way back: distill_backward in place, reduce_scatter
                   of y's gradient, layer_norm_backward, combine_backward,
                   route_backward with balance_backward on top, layer_norm_backward,
                   all_gather, embedding_backward on top of the logits' part
  clipping         all_reduce of what every rank has, the global norm, plain
                   gradient descent

    python examples/distill_step.py --steps 5
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import copy_reduce_snac_amd as snac  # noqa: E402
from copy_reduce_snac_amd import operators as ops  # noqa: E402
from copy_reduce_snac_amd import tensors as coll  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROUTER = dict(score="softmax", renorm=True)


class DistillStep:
    def __init__(self, ranks=4, tokens=256, width=256, vocab=4096, experts=8, topk=2, choices=16, temperature=2.0,
                 balance=0.05, seed=0):
        if vocab % ranks:  # a column that no rank held would be a choice without a logit
            raise ValueError(f"vocab {vocab} is not a multiple of ranks {ranks}: the shards are equal")
        self.n, self.tokens, self.width, self.topk, self.experts = ranks, tokens, width, topk, experts
        self.local, self.vocab, self.temperature, self.balance = vocab // ranks, vocab, temperature, balance
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, scale=1.0, dtype=F32):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

        self.tables = [normal(self.local, width, scale=width ** -0.5, dtype=BF16) for _ in range(ranks)]
        self.router = normal(width, experts, scale=2 * width ** -0.5)
        self.matrices = normal(experts, width, width, scale=width ** -0.5, dtype=BF16)
        self.norms = [1.0 + normal(width, scale=0.1), normal(width, scale=0.1), 1.0 + normal(width, scale=0.1),
                      normal(width, scale=0.1)]  # weight and bias of the two
        self.ids = [torch.randint(0, vocab, (tokens,), generator=g, device="cuda") for _ in range(ranks)]
        every = ranks * tokens
        self.chosen = torch.stack([torch.randperm(vocab, generator=g, device="cuda")[:choices] for _ in range(every)])
        self.chosen[::17] = -1  # padding tokens
        self.teacher = normal(every, choices, scale=2.0).sort(dim=1, descending=True).values.contiguous()
        # gradients, in places that do not change: the norm's list is made once
        self.dtables = [torch.empty(self.local, width, device="cuda") for _ in range(ranks)]
        self.drouter = self.each(width, experts)
        self.dmatrices = self.each(experts, width, width)
        self.dnorms = self.each(4, width)
        self.norm = torch.empty(1, device="cuda")
        self.grads = ops.GradList(self.dtables + self.drouter[:1] + self.dmatrices[:1] + self.dnorms[:1])
        self.handle = snac.snac_init(ranks)

    def close(self):
        self.grads.close()
        snac.snac_finalize(self.handle)

    def each(self, *shape, dtype=F32):
        return [torch.empty(*shape, dtype=dtype, device="cuda") for _ in range(self.n)]

    def forward_backward(self):
        n, t, w, k, e, v = self.n, self.tokens, self.width, self.topk, self.experts, self.local
        tau, whole = self.temperature, dict(vocab=self.vocab, temperature=self.temperature)
        w1, b1, w2, b2 = self.norms
        every = torch.cat(self.ids)
        part, x = self.each(n * t, w, dtype=BF16), self.each(t, w, dtype=BF16)
        for r in range(n):
            ops.embedding(self.tables[r], every, part[r], first=r * v, scale=w ** 0.5)
        coll.reduce_scatter(part, x, self.handle)

        # experts
        h, stats1 = self.each(t, w, dtype=BF16), self.each(t, 2)
        weights, ids, loads = self.each(t, k), self.each(t, k, dtype=I32), self.each(2, e)
        counts, rows, slots = self.each(e, dtype=I32), self.each(t, k, dtype=I32), self.each(t * k, dtype=I32)
        sent, made = self.each(t * k, w, dtype=BF16), self.each(t * k, w, dtype=BF16)
        mixed, logits = self.each(t, w, dtype=BF16), []
        for r in range(n):
            ops.layer_norm(x[r], w1, b1, h[r], stats=stats1[r])
            logits.append(h[r].float() @ self.router)
            ops.route(logits[r], weights[r], ids[r], **ROUTER)
            ops.balance_load(logits[r], ids[r], loads[r], self.handle)
            ops.dispatch_plan(ids[r], counts[r], rows[r], slots[r], self.handle)
            ops.dispatch(h[r], rows[r], sent[r])
        coll.all_reduce(loads, loads, self.handle)
        uneven = torch.empty(1, device="cuda")
        ops.balance_loss(loads[0], uneven, coefficient=self.balance)
        by_expert = torch.stack(counts).tolist()
        for r in range(n):
            at = 0
            for i, m in enumerate(by_expert[r]):
                torch.mm(sent[r][at:at + m], self.matrices[i], out=made[r][at:at + m])
                at += m
            ops.combine(made[r], rows[r], weights[r], mixed[r])

        # logits by shards of the vocabulary, and what they are off by
        s = [x[r] + mixed[r] for r in range(n)]
        y, stats2, ys = self.each(t, w, dtype=BF16), self.each(t, 2), self.each(n * t, w, dtype=BF16)
        for r in range(n):
            ops.layer_norm(s[r], w2, b2, y[r], stats=stats2[r])
        coll.all_gather(y, ys, self.handle)
        z = [ys[r] @ self.tables[r].t() for r in range(n)]
        parts, joint = self.each(n * t, 4), self.each(n, n * t, 4)
        loss, stats = self.each(n * t), self.each(n * t, 2)
        for r in range(n):
            ops.distill_shard(z[r], self.chosen, self.teacher, parts[r], first=r * v, **whole)
        coll.all_gather(parts, joint, self.handle)
        for r in range(n):
            ops.distill_join(joint[r], self.chosen, self.teacher, loss[r], stats[r], **whole)
        scale = tau * tau / (n * t)
        total = loss[0].sum() * scale + uneven[0]

        # backward: logits and the table's part in them
        dys, dy = self.each(n * t, w, dtype=BF16), self.each(t, w, dtype=BF16)
        for r in range(n):
            ops.distill_backward(z[r], self.chosen, self.teacher, stats[r], z[r], scale=scale, first=r * v, **whole)
            torch.mm(z[r], self.tables[r], out=dys[r])
            torch.mm(z[r].float().t(), ys[r].float(), out=self.dtables[r])
        coll.reduce_scatter(dys, dy, self.handle)

        # experts
        dx = self.each(t, w, dtype=BF16)
        for r in range(n):
            dn = self.dnorms[r]
            ds = torch.empty_like(dy[r])
            ops.layer_norm_backward(dy[r], s[r], w2, stats2[r], ds, dn[2], dn[3], self.handle)
            dmade, dweights = torch.zeros_like(made[r]), torch.empty_like(weights[r])
            ops.combine_backward(ds, made[r], rows[r], weights[r], dmade, dweights)
            dsent, at = torch.zeros_like(sent[r]), 0
            for i, m in enumerate(by_expert[r]):
                g = dmade[at:at + m]
                torch.mm(g, self.matrices[i].t(), out=dsent[at:at + m])
                torch.mm(sent[r][at:at + m].float().t(), g.float(), out=self.dmatrices[r][i])
                at += m
            dh, dlogits = torch.empty_like(h[r]), torch.empty_like(logits[r])
            ops.combine(dsent, rows[r], None, dh)
            ops.route_backward(logits[r], ids[r], dweights, dlogits, **ROUTER)
            ops.balance_backward(logits[r], ids[r], loads[r], dlogits, coefficient=self.balance, accumulate=True)
            torch.mm(h[r].float().t(), dlogits, out=self.drouter[r])
            dh += (dlogits @ self.router.t()).to(BF16)
            ops.layer_norm_backward(dh, x[r], w1, stats1[r], dh, dn[0], dn[1], self.handle)
            torch.add(ds, dh, out=dx[r])
        dxs = self.each(n * t, w, dtype=BF16)
        coll.all_gather(dx, dxs, self.handle)
        for r in range(n):
            ops.embedding_backward(dxs[r], every, self.dtables[r], self.handle, first=r * v, scale=w ** 0.5, accumulate=True)
        for grads in (self.drouter, self.dmatrices, self.dnorms):
            coll.all_reduce(grads, grads, self.handle)
        return total, ids

    def step(self, rate=0.2, max_norm=1.0):
        loss, _ = self.forward_backward()
        ops.clip_grad_norm(self.grads, max_norm, self.norm)
        for r in range(self.n):
            self.tables[r].sub_((self.dtables[r] * rate).to(BF16))
        self.router.sub_(self.drouter[0] * rate)
        self.matrices.sub_((self.dmatrices[0] * rate).to(BF16))
        for p, g in zip(self.norms, self.dnorms[0]):
            p.sub_(g * rate)
        return loss


def main(argv=None) -> list[float]:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--tokens", type=int, default=256)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--vocab", type=int, default=4096)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args(argv)
    torch.cuda.set_device(0)
    m = DistillStep(a.ranks, a.tokens, a.width, a.vocab)
    losses = []
    try:
        for i in range(a.steps):
            loss = m.step()
            snac.snac_check(m.handle)
            losses.append(float(loss))
            print(f"step {i}: loss {losses[-1]:.4f}, gradient norm {float(m.norm):.4f}", flush=True)
    finally:
        m.close()
    return losses


if __name__ == "__main__":
    main()
