"""Sums of the embedding gradient over long runs of one token on the GPU.

Bounds (u = 2^-24): the rows of a chunk are added without error (binary64, or
bf16 rows of nearly one magnitude in binary32), each chunk's sum is rounded to
binary32 once, the chunks are joined in binary64 (n 2^-52 of the magnitudes at
most) and the result is rounded once: (2 u + n 2^-52) of the sum of
magnitudes, whatever the run's length.  Small whole numbers have no error."""
from __future__ import annotations

import pytest

from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24
DT = {"f32": "float32", "bf16": "bfloat16"}


def ops():
    from copy_reduce_snac_amd import operators

    return operators


@pytest.fixture(scope="module")
def torch():
    import torch

    torch.cuda.set_device(0)
    return torch


@pytest.fixture(scope="module")
def handle(torch):
    import copy_reduce_snac_amd as snac

    h = snac.snac_init(2)
    yield h
    snac.snac_finalize(h)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens", [3000, 30000, 300000, 2 ** 22])
def test_error_does_not_grow_with_the_run(torch, handle, dtype, accumulate, tokens):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    d = (0.5 + torch.rand(tokens, 12, generator=g, device="cuda")).to(getattr(torch, DT[dtype]))
    d[:, 3] = d[0, 3]  # every row the same: the errors of a binary32 sum all point one way
    dt = torch.full((2, 12), 0.375 if accumulate else 77.0, device="cuda")
    ops().embedding_backward(d, torch.ones(tokens, dtype=torch.int64, device="cuda"), dt, handle, scale=0.75,
                             accumulate=accumulate)
    want = 0.75 * d.double().sum(0) + (0.375 if accumulate else 0.0)
    assert bool((dt[0] == (0.375 if accumulate else 0.0)).all())
    err = ((dt[1].double() - want).abs() / want).max().item()
    assert err <= 2 * U + tokens * 2.0 ** -52, err


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens", [33, 600, 4096, 4097, 8192, 8193, 70001])
@pytest.mark.parametrize("names", [1, 3])
def test_whole_numbers_are_exact(torch, handle, dtype, accumulate, tokens, names):
    """Rows that differ, so that one lost, doubled or put to another token shows; runs over more than 64 chunks."""
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens + names)
    vocab, width = 5, 70
    d = torch.randint(-8, 9, (tokens, width), generator=g, device="cuda").to(getattr(torch, DT[dtype]))
    ids = 1 + torch.randint(0, names, (tokens,), generator=g, device="cuda")
    before = torch.randint(-99, 99, (vocab, width), generator=g, device="cuda").float()
    dt = before.clone()
    ops().embedding_backward(d, ids, dt, handle, accumulate=accumulate)
    want = torch.zeros(vocab, width, dtype=torch.float64, device="cuda").index_add_(0, ids, d.double())
    assert float(want.abs().max()) < 2 ** 23
    assert torch.equal(dt.double(), want + before.double() if accumulate else want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [70, 2048])
@pytest.mark.parametrize("tokens", [5, 200])
def test_accumulating_rounds_once(torch, handle, dtype, width, tokens):
    """What is there takes the rounded product away: what rounding left out stays, and that is representable.  One row
    of the token is not zero, so runs inside a chunk and over several give its product alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    d = torch.zeros(tokens, width, dtype=getattr(torch, DT[dtype]), device="cuda")
    d[1] = torch.randn(width, generator=g, device="cuda").to(d.dtype)
    scale = float(torch.tensor(0.7).item())
    product = d[1].double() * scale
    dt = -product.float().expand(3, width).contiguous()
    old = dt.clone()
    ops().embedding_backward(d, torch.full((tokens,), 2, device="cuda"), dt, handle, scale=scale, accumulate=True)
    left = product + old[2].double()
    assert int((left != 0).sum()) > width // 2
    assert torch.equal(dt[2].double(), left) and torch.equal(dt[:2], old[:2])
