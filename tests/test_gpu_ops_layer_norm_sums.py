"""The sums over tokens of layer norm's gradient: binary32 goes no further than
32 tokens.  Numbers that binary64 adds up exactly and binary32 does not: whole
numbers, 2^24 and -2^24 among ones, at most one of the large ones within 32
tokens that a lane takes.  The workgroups' sums are small whole numbers, so
their roundings are exact too, and so is the result."""
from __future__ import annotations

import pytest

from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DT = {"f32": "float32", "bf16": "bfloat16"}
BIG = 2.0 ** 24


@pytest.fixture(scope="module")
def torch():
    import torch

    torch.cuda.set_device(0)
    return torch


@pytest.fixture(scope="module")
def ops(torch):
    from copy_reduce_snac_amd import operators

    return operators


@pytest.fixture(scope="module")
def handle(torch):
    import copy_reduce_snac_amd as snac

    h = snac.snac_init(1)
    yield h
    snac.snac_finalize(h)


# rows that go side by side in a workgroup: 64 of up to 256 bytes, 32, 16, 8, 4
SIDE = [("f32", 60, 64), ("bf16", 128, 64), ("bf16", 127, 64), ("f32", 128, 32), ("bf16", 250, 32), ("f32", 256, 16), ("bf16", 1000, 16),
        ("f32", 513, 8), ("bf16", 2048, 8), ("bf16", 2051, 4), ("f32", 2000, 4)]


@pytest.mark.parametrize("groups", [1, 200])
@pytest.mark.parametrize("dtype,width,side", SIDE)
def test_rows_side_by_side(torch, ops, handle, dtype, width, side, groups):
    """One turn of one workgroup, and of 200."""
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    # half of a workgroup's rows are large and cancel, the others are 1; the order is another in each
    row = torch.ones(side, device="cuda")
    row[:side // 2:2], row[1:side // 2:2] = BIG, -BIG
    v = torch.stack([row[torch.randperm(side, generator=g, device="cuda")] for _ in range(groups)]).flatten()
    tokens = side * groups
    dout = v.unsqueeze(1).repeat(1, width).to(getattr(torch, DT[dtype]))
    x = torch.ones_like(dout)  # h is 1: both sums are dout's
    x[:, ::2] = -1
    stats = torch.tensor([0.0, 1.0], device="cuda").repeat(tokens, 1)
    dx, dw, db = torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    ops.layer_norm_backward(dout, x, None, stats, dx, dw, db, handle)
    want = torch.full((width,), float(groups * (side // 2)), device="cuda")
    assert torch.equal(db, want), (db.min(), db.max(), want[0])
    assert torch.equal(dw, want * x[0].float())
    ops.layer_norm_backward(dout, x, None, stats, dx, dw, db, handle, accumulate=True)
    assert torch.equal(db, 2 * want) and torch.equal(dw, 2 * want * x[0].float())


# rows that a workgroup takes one at a time, rows side by side, and (36 KiB) those of which a workgroup takes columns
@pytest.mark.parametrize("dtype,width,side,groups", [("bf16", 16384, 1, 256), ("f32", 5003, 1, 256), ("bf16", 3000, 4, 256),
                                                     ("f32", 64, 64, 256), ("f32", 9216, 0, 114)])
def test_more_than_32_turns(torch, ops, handle, dtype, width, side, groups):
    """2^24, then nothing, after 32 turns ones and at the end -2^24: 40 turns of the workgroups that fill the chip."""
    v = torch.zeros(40, groups * max(side, 1), device="cuda")
    v[0], v[32:39], v[39] = BIG, 1.0, -BIG
    if side == 0:  # the rows of a workgroup follow one another there
        v = v.t()
    tokens = v.numel()
    dout = v.reshape(tokens, 1).repeat(1, width).to(getattr(torch, DT[dtype]))
    x = torch.ones_like(dout)
    stats = torch.tensor([0.0, 1.0], device="cuda").repeat(tokens, 1)
    dx, dw, db = torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    want = torch.full((width,), 7.0 * tokens / 40, device="cuda")
    for _ in range(2):  # the scratch of one call does not matter to the next
        ops.layer_norm_backward(dout, x, None, stats, dx, dw, db, handle)
        assert torch.equal(db, want) and torch.equal(dw, want), (db.min(), db.max(), want[0])
    ops.layer_norm_backward(dout, x, None, stats, dx, dw, None, handle, accumulate=True)
    assert torch.equal(dw, 2 * want)


@pytest.mark.parametrize("dtype,width,tokens", [("bf16", 16384, 32768), ("bf16", 12288, 40001), ("bf16", 8192, 131072), ("f32", 16384, 16384)])
def test_many_tokens_on_a_default_context(torch, ops, handle, dtype, width, tokens):
    """The partial sums' scratch does not grow with the tokens: whole numbers come out whole."""
    dt = getattr(torch, DT[dtype])
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    x, dout = (torch.randint(-2, 3, (tokens, width), generator=g, device="cuda", dtype=torch.int8).to(dt) for _ in "xd")
    stats = torch.tensor([0.0, 1.0], device="cuda").repeat(tokens, 1)
    dx, dw, db = torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    ops.layer_norm_backward(dout, x, None, stats, dx, dw, db, handle)
    want_w, want_b = torch.zeros(width, device="cuda"), torch.zeros(width, device="cuda")
    for t in range(0, tokens, 4096):  # sums below 2^24, exact
        want_b += dout[t:t + 4096].sum(0, dtype=torch.float32)
        want_w += (dout[t:t + 4096] * x[t:t + 4096]).sum(0, dtype=torch.float32)
    assert torch.equal(dw, want_w) and torch.equal(db, want_b)
    for t in (0, tokens // 2, tokens - 1):
        one = torch.empty_like(dx[:1])
        ops.layer_norm_backward(dout[t:t + 1], x[t:t + 1], None, stats[t:t + 1], one, None, None, handle)
        assert torch.equal(one[0], dx[t]), t


# rows that 2, 4, 8 and 16 waves hold, and one that a workgroup reads several times
@pytest.mark.parametrize("dtype,width", [("f32", 1024), ("f32", 2048), ("f32", 4096), ("f32", 8192), ("f32", 16384), ("bf16", 2048),
                                         ("bf16", 4096), ("bf16", 8192), ("bf16", 16384), ("bf16", 32768)])
def test_a_rows_sums_over_its_waves(torch, ops, handle, dtype, width):
    """A row's sums are binary64 over its units, those of different waves as well: 2^30 in one unit, ones in the others and
    -2^30 in a unit of the last wave have their exact sum.  h is 0 and 1 / deviation 1, so dx is dout less its mean,
    exact in binary32 where dout is 1."""
    n = 16 // (4 if dtype == "f32" else 2)  # a unit's elements
    dout = torch.ones(6, width, device="cuda")
    for r, (a, b) in enumerate([(0, width // n - 1), (3, width // n - 2), (width // n // 2, width // n - 5)]):
        for row, first in ((r, 2.0 ** 30), (r + 3, -2.0 ** 30)):
            dout[row, a * n:(a + 1) * n] = 0
            dout[row, b * n:(b + 1) * n] = 0
            dout[row, a * n], dout[row, b * n] = first, -first
    dout = dout.to(getattr(torch, DT[dtype]))
    x, stats = torch.full_like(dout, 3.0), torch.tensor([3.0, 1.0], device="cuda").repeat(6, 1)
    dx = torch.empty_like(dout)
    ops.layer_norm_backward(dout, x, None, stats, dx, None, None, handle)
    g = dout.double()
    want = (g - g.mean(dim=1, keepdim=True)).float().to(dout.dtype)
    assert torch.equal(dx, want), (dx.float()[:, 100], want.float()[:, 100])


def test_several_launches_in_a_graph(torch, ops, handle):
    """Two launches and their joins, captured and replayed with other inputs, eager calls of the same scratch between."""
    tokens, width = 8300, 16384
    g = torch.Generator(device="cuda")
    x, dout = (torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda") for _ in "xd")
    stats = torch.tensor([0.0, 1.0], device="cuda").repeat(tokens, 1)
    dx, dw, db = torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")

    def fill(seed):
        g.manual_seed(seed)
        x.normal_(generator=g)
        dout.normal_(generator=g)

    def run():
        ops.layer_norm_backward(dout, x, None, stats, dx, dw, db, handle)

    wants = {}
    for seed in (1, 2, 3):
        fill(seed)
        run()
        torch.cuda.synchronize()
        wants[seed] = [t.clone() for t in (dx, dw, db)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for seed in (1, 2, 3, 2):
        small = torch.empty(width, device="cuda")  # another call of the scratch, a sum of few rows
        ops.layer_norm_backward(dout[:700], x[:700], None, stats[:700], dx[:700], small, None, handle)
        fill(seed)
        for t in (dx, dw, db):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, want, name in zip((dx, dw, db), wants[seed], ("dx", "dw", "db")):
            assert torch.equal(got, want), (seed, name)
