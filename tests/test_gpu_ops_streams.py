"""The operators on side streams and in HIP graphs: a graph of a step around
the collectives is captured once and replayed with new inputs, the program's
own eager work between the replays, each replay held against the eager
result."""
from __future__ import annotations

import pytest

from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

TOKENS, EXPERTS, TOPK, WIDTH, VOCAB = 3000, 64, 4, 264, 700


class Step:
    """Every operator once, on buffers of its own."""

    def __init__(self, torch, handle, ops):
        self.torch, self.handle, self.ops = torch, handle, ops
        bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
        m = TOKENS * TOPK
        e = lambda *s, dtype=f32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.tokens = e(TOKENS, dtype=torch.int64)
        self.table = e(VOCAB, WIDTH, dtype=bf)
        self.logits, self.bias = e(TOKENS, EXPERTS), e(EXPERTS)
        self.dout = e(TOKENS, WIDTH, dtype=bf)
        self.out = dict(x=e(TOKENS, WIDTH, dtype=bf), weights=e(TOKENS, TOPK), ids=e(TOKENS, TOPK, dtype=i32),
                        counts=e(EXPERTS, dtype=i32), rows=e(TOKENS, TOPK, dtype=i32), slots=e(m, dtype=i32),
                        sent=e(m, WIDTH, dtype=bf), y=e(TOKENS, WIDTH, dtype=bf), dsent=e(m, WIDTH, dtype=bf),
                        dweights=e(TOKENS, TOPK), dlogits=e(TOKENS, EXPERTS), dx=e(TOKENS, WIDTH, dtype=bf),
                        dtable=e(VOCAB, WIDTH), clipped=e(VOCAB, WIDTH), norm=e(1))
        self.list = ops.GradList([self.out["dtable"]], [self.out["clipped"]])

    def fill(self, seed):
        g = self.torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.tokens.random_(0, VOCAB, generator=g)
        for t in (self.table, self.logits, self.dout):
            t.normal_(generator=g)
        self.bias.normal_(0.0, 0.1, generator=g)

    def run(self):
        o, p = self.out, self.ops
        kw = dict(score="sigmoid", renorm=True, scale=2.5)
        p.embedding(self.table, self.tokens, o["x"], scale=2.0)
        p.route(self.logits, o["weights"], o["ids"], bias=self.bias, groups=8, topk_groups=3, **kw)
        p.dispatch_plan(o["ids"], o["counts"], o["rows"], o["slots"], self.handle)
        p.dispatch(o["x"], o["rows"], o["sent"])
        p.combine(o["sent"], o["rows"], o["weights"], o["y"])
        p.combine_backward(self.dout, o["sent"], o["rows"], o["weights"], o["dsent"], o["dweights"])
        p.route_backward(self.logits, o["ids"], o["dweights"], o["dlogits"], **kw)
        p.combine(o["dsent"], o["rows"], None, o["dx"])
        p.embedding_backward(o["dx"], self.tokens, o["dtable"], self.handle, scale=2.0)
        p.clip_grad_norm(self.list, 1.0, o["norm"])

    def copy(self):
        return {k: v.clone() for k, v in self.out.items()}


@pytest.fixture(scope="module")
def step():
    import torch

    import copy_reduce_snac_amd as snac
    from copy_reduce_snac_amd import operators

    torch.cuda.set_device(0)
    h = snac.snac_init(1)
    s = Step(torch, h, operators)
    yield s
    s.list.close()
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
    same(step, eager(step, 1), "first")
    want = eager(step, 1)
    eager(step, 2)
    eager(step, 1)
    same(step, want, "again")


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
