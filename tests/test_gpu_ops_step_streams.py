"""Layer norm, the balance loss and distillation on side streams and in HIP
graphs: a graph of them all is captured once and replayed with new inputs, the
program's own eager work between the replays, each replay held against the
eager result."""
from __future__ import annotations

import pytest

from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

TOKENS, EXPERTS, TOPK, WIDTH, VOCAB, CHOICES = 2500, 64, 4, 520, 3001, 20


class Step:
    """Every operator once, on buffers of its own."""

    def __init__(self, torch, handle, ops):
        self.torch, self.handle, self.ops = torch, handle, ops
        bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
        e = lambda *s, dtype=f32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.x, self.dout = e(TOKENS, WIDTH, dtype=bf), e(TOKENS, WIDTH, dtype=bf)
        self.weight, self.bias = e(WIDTH), e(WIDTH)
        self.logits, self.z = e(TOKENS, EXPERTS), e(TOKENS, VOCAB, dtype=bf)
        self.ids, self.teacher = e(TOKENS, CHOICES, dtype=torch.int64), e(TOKENS, CHOICES)
        self.dloss = e(TOKENS)
        cut = self.cut = VOCAB // 2
        self.out = dict(y=e(TOKENS, WIDTH, dtype=bf), stats=e(TOKENS, 2), dx=e(TOKENS, WIDTH, dtype=bf), dw=e(WIDTH),
                        db=e(WIDTH), weights=e(TOKENS, TOPK), chosen=e(TOKENS, TOPK, dtype=i32), load=e(2, EXPERTS), balance=e(1),
                        dlogits=e(TOKENS, EXPERTS), loss=e(TOKENS), zstats=e(TOKENS, 2), dz=e(TOKENS, VOCAB, dtype=bf),
                        parts=e(2, TOKENS, 4), loss2=e(TOKENS), zstats2=e(TOKENS, 2), dz2=e(TOKENS, VOCAB - cut, dtype=bf))

    def fill(self, seed):
        g = self.torch.Generator(device="cuda")
        g.manual_seed(seed)
        for t in (self.x, self.dout, self.weight, self.bias, self.logits, self.z, self.teacher, self.dloss):
            t.normal_(generator=g)
        self.ids.random_(-1, VOCAB, generator=g)

    def run(self):
        o, p, cut = self.out, self.ops, self.cut
        kw = dict(vocab=VOCAB, temperature=1.5)
        p.layer_norm(self.x, self.weight, self.bias, o["y"], stats=o["stats"])
        p.layer_norm_backward(self.dout, self.x, self.weight, o["stats"], o["dx"], o["dw"], o["db"], self.handle)
        p.route(self.logits, o["weights"], o["chosen"])
        p.balance_load(self.logits, o["chosen"], o["load"], self.handle)
        p.balance_loss(o["load"], o["balance"])
        p.balance_backward(self.logits, o["chosen"], o["load"], o["dlogits"], dloss=o["balance"])
        p.distill(self.z, self.ids, self.teacher, o["loss"], o["zstats"], temperature=1.5)
        p.distill_backward(self.z, self.ids, self.teacher, o["zstats"], o["dz"], dloss=self.dloss, temperature=1.5)
        p.distill_shard(self.z[:, :cut], self.ids, self.teacher, o["parts"][0], first=0, **kw)
        p.distill_shard(self.z[:, cut:], self.ids, self.teacher, o["parts"][1], first=cut, **kw)
        p.distill_join(o["parts"], self.ids, self.teacher, o["loss2"], o["zstats2"], **kw)
        p.distill_backward(self.z[:, cut:], self.ids, self.teacher, o["zstats2"], o["dz2"], first=cut, **kw)
        # the same scratch again, within a call of the next use
        p.layer_norm_backward(o["dx"], self.x, None, o["stats"], o["dx"], o["dw"], None, self.handle, accumulate=True)

    def copy(self):
        return {k: v.clone() for k, v in self.out.items()}


@pytest.fixture(scope="module")
def step():
    import torch

    import copy_reduce_snac_amd as snac
    from copy_reduce_snac_amd import operators

    torch.cuda.set_device(0)
    h = snac.snac_init(1)
    yield Step(torch, h, operators)
    snac.snac_finalize(h)


def eager(step, seed):
    step.fill(seed)
    step.run()
    step.torch.cuda.synchronize()
    return step.copy()


def same(step, want, what):
    for k, v in step.out.items():
        assert step.torch.equal(v, want[k]), f"{what}: {k}"


def test_same_bits_twice(step):
    want = eager(step, 1)
    eager(step, 2)
    eager(step, 1)
    same(step, want, "again")
    assert all(bool(v.float().isfinite().all()) for v in want.values())


def test_on_a_side_stream(step):
    want = eager(step, 3)
    eager(step, 4)
    s = step.torch.cuda.Stream()
    s.wait_stream(step.torch.cuda.current_stream())
    with step.torch.cuda.stream(s):
        step.fill(3)
        step.run()
    s.synchronize()
    same(step, want, "side stream")


def test_graph_replays(step):
    torch = step.torch
    wants = {seed: eager(step, seed) for seed in (5, 6, 7, 8)}
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step.fill(5)
        step.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step.run()
    for seed in (5, 6, 7, 8, 6):
        step.fill(seed)                       # eager work between the replays
        for v in step.out.values():
            v.zero_()
        torch.randn(1000, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        same(step, wants[seed], f"replay of {seed}")


def test_two_contexts_at_once(step):
    """Calls on two streams do not share scratch when each has a context of its own."""
    import copy_reduce_snac_amd as snac

    torch = step.torch
    other = snac.snac_init(1)
    try:
        two = Step(torch, other, step.ops)
        want = eager(step, 9)
        two.fill(10)
        two.run()
        torch.cuda.synchronize()
        want2 = two.copy()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            for v in (*step.out.values(), *two.out.values()):
                v.zero_()
            for one, s in zip((step, two), streams):
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    one.run()
            torch.cuda.synchronize()
            same(step, want, "first stream")
            same(two, want2, "second stream")
    finally:
        torch.cuda.synchronize()
        snac.snac_finalize(other)
