"""Training steps of a small mixture-of-experts layer over N logical ranks:
the operators of ``copy_reduce_snac_amd.operators`` around the collectives of
``copy_reduce_snac_amd.tensors``.

Rank r holds a shard of the vocabulary, a shard of the experts and tokens of
its own.  One step:

  embedding        every shard looks up all ranks' tokens; reduce_scatter sums
                   the shards and leaves each rank its tokens' rows
  route            scores, groups, top-k
  dispatch         rows packed by expert; all_to_all_v to the experts' ranks
  experts          one matrix a expert (torch)
  combine          all_to_all_v back, the weighted sum, a squared error
  backward         combine_backward, all_to_all_v both ways, route_backward,
                   all_gather of the rows' gradients, embedding_backward
  clipping         all_reduce of the router's gradient, the global norm over
                   every rank's gradients, plain gradient descent

    python examples/moe_step.py --steps 5
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


class MoeStep:
    def __init__(self, ranks=4, tokens=512, width=256, vocab=4096, experts=32, topk=4, groups=4, topk_groups=2, seed=0):
        self.n, self.tokens, self.width, self.topk = ranks, tokens, width, topk
        self.experts, self.groups, self.topk_groups = experts, groups, topk_groups
        self.vocab, self.local = vocab // ranks, experts // ranks
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, scale=1.0, dtype=F32):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

        self.tables = [normal(self.vocab, width, scale=0.05, dtype=BF16) for _ in range(ranks)]
        self.router = normal(width, experts, scale=0.3)
        self.bias = normal(experts, scale=0.02)
        self.weights = [normal(self.local, width, width, scale=width ** -0.5, dtype=BF16) for _ in range(ranks)]
        self.ids = [torch.randint(0, vocab, (tokens,), generator=g, device="cuda") for _ in range(ranks)]
        self.target = [normal(tokens, width) for _ in range(ranks)]
        # gradients, in places that do not change: the norm's list is made once
        self.dtables = [torch.empty(self.vocab, width, device="cuda") for _ in range(ranks)]
        self.dweights = [torch.empty(self.local, width, width, device="cuda") for _ in range(ranks)]
        self.drouter = [torch.empty(width, experts, device="cuda") for _ in range(ranks)]
        self.norm = torch.empty(1, device="cuda")
        self.grads = ops.GradList(self.dtables + self.dweights + self.drouter[:1])
        self.handle = snac.snac_init(ranks)

    def close(self):
        self.grads.close()
        snac.snac_finalize(self.handle)

    def each(self, *shape, dtype=F32):
        return [torch.empty(*shape, dtype=dtype, device="cuda") for _ in range(self.n)]

    def exchange(self, rows, counts, sizes):
        """all_to_all_v of packed rows; counts[s][d] rows, sizes[d] rows received."""
        out = [torch.empty(m, self.width, dtype=BF16, device="cuda") for m in sizes]
        w = self.width
        coll.all_to_all_v(rows, out, [[c * w for c in row] for row in counts], self.handle)
        return out

    def pieces(self, rank, counts):
        """(first row, rows, local expert) of what rank `rank` received: by source, then by expert."""
        at = 0
        for s in range(self.n):
            for e in range(self.local):
                n = counts[s][rank * self.local + e]
                yield at, n, e
                at += n

    def forward_backward(self, scale=2.5):
        n, t, w, k = self.n, self.tokens, self.width, self.topk
        kw = dict(score="sigmoid", renorm=True, scale=scale)
        every = torch.cat(self.ids)
        part = self.each(n * t, w, dtype=BF16)
        x = self.each(t, w, dtype=BF16)
        for r in range(n):
            ops.embedding(self.tables[r], every, part[r], first=r * self.vocab, scale=w ** 0.5)
        coll.reduce_scatter(part, x, self.handle)

        logits = [v.float() @ self.router for v in x]
        wts, ids = self.each(t, k), self.each(t, k, dtype=I32)
        counts, rows, slots = self.each(self.experts, dtype=I32), self.each(t, k, dtype=I32), self.each(t * k, dtype=I32)
        sent = self.each(t * k, w, dtype=BF16)
        for r in range(n):
            ops.route(logits[r], wts[r], ids[r], bias=self.bias, groups=self.groups, topk_groups=self.topk_groups, **kw)
            ops.dispatch_plan(ids[r], counts[r], rows[r], slots[r], self.handle)
            ops.dispatch(x[r], rows[r], sent[r])
        by_expert = torch.stack(counts).tolist()  # the one wait for the device: the exchange's counts are host values
        there = [[sum(c[d * self.local:(d + 1) * self.local]) for d in range(n)] for c in by_expert]
        back = [list(c) for c in zip(*there)]
        received = self.exchange(sent, there, [sum(there[s][d] for s in range(n)) for d in range(n)])
        made = [torch.empty_like(v) for v in received]
        for r in range(n):
            for at, m, e in self.pieces(r, by_expert):
                torch.mm(received[r][at:at + m], self.weights[r][e], out=made[r][at:at + m])
        y = self.exchange(made, back, [t * k] * n)
        out = self.each(t, w, dtype=BF16)
        for r in range(n):
            ops.combine(y[r], rows[r], wts[r], out[r])
        error = [out[r].float() - self.target[r] for r in range(n)]
        loss = sum((v * v).sum() for v in error) / (2 * n * t)

        dout = [(v / (n * t)).to(BF16) for v in error]
        dy, dwts = [torch.zeros_like(v) for v in y], self.each(t, k)
        for r in range(n):
            ops.combine_backward(dout[r], y[r], rows[r], wts[r], dy[r], dwts[r])
        dmade = self.exchange(dy, there, [v.shape[0] for v in made])
        dreceived = [torch.empty_like(v) for v in received]
        for r in range(n):
            self.dweights[r].zero_()
            for at, m, e in self.pieces(r, by_expert):
                g = dmade[r][at:at + m]
                torch.mm(g, self.weights[r][e].t(), out=dreceived[r][at:at + m])
                self.dweights[r][e] += received[r][at:at + m].float().t() @ g.float()
        dsent = self.exchange(dreceived, back, [t * k] * n)
        dx = self.each(t, w, dtype=BF16)
        for r in range(n):
            dlogits = torch.empty_like(logits[r])
            ops.combine(dsent[r], rows[r], None, dx[r])
            ops.route_backward(logits[r], ids[r], dwts[r], dlogits, **kw)
            torch.mm(x[r].float().t(), dlogits, out=self.drouter[r])
            dx[r] += (dlogits @ self.router.t()).to(BF16)
        all_dx = self.each(n * t, w, dtype=BF16)
        coll.all_gather(dx, all_dx, self.handle)
        for r in range(n):
            ops.embedding_backward(all_dx[r], every, self.dtables[r], self.handle, first=r * self.vocab, scale=w ** 0.5)
        coll.all_reduce(self.drouter, self.drouter, self.handle)
        return loss, ids

    def step(self, rate=0.5, max_norm=1.0):
        loss, _ = self.forward_backward()
        ops.clip_grad_norm(self.grads, max_norm, self.norm)
        for r in range(self.n):
            self.tables[r].sub_((self.dtables[r] * rate).to(BF16))
            self.weights[r].sub_((self.dweights[r] * rate).to(BF16))
        self.router.sub_(self.drouter[0] * rate)
        return loss


def main(argv=None) -> list[float]:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args(argv)
    torch.cuda.set_device(0)
    m = MoeStep(a.ranks, a.tokens, a.width, experts=a.experts)
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
