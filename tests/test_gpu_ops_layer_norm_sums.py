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
