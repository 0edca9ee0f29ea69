"""The gradient of the combine's weights over wide rows on the GPU.

Bound (u = 2^-24): the products of a 16-byte unit are added in binary32 with
fused multiply-adds, one rounding each (4 or 8 of them), the units in binary64,
and the sum is rounded once: 5 or 9 u of the sum of magnitudes (here the sum
itself: all positive), whatever the width."""
from __future__ import annotations

import pytest

from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24


@pytest.mark.parametrize("dtype,terms", [("float32", 4), ("bfloat16", 8)])
@pytest.mark.parametrize("width", [2048, 8192, 8195, 65536, 200001])
def test_error_does_not_grow_with_the_width(dtype, terms, width):
    import torch

    from copy_reduce_snac_amd import operators as ops

    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    tokens, topk = 6, 2
    dout = torch.ones(tokens, width, device="cuda")
    dout[3:] = 0.5 + torch.rand(3, width, generator=g, device="cuda")
    y = torch.tensor([0.1, 0.3, 0.7, 1 / 3], device="cuda").repeat(3)[:, None].expand(12, width).contiguous()
    y[7:] *= 0.5 + torch.rand(5, width, generator=g, device="cuda")
    dout, y = dout.to(getattr(torch, dtype)), y.to(getattr(torch, dtype))
    rows = torch.arange(12, dtype=torch.int32, device="cuda").flip(0).view(tokens, topk).contiguous()
    w, dw = torch.ones(tokens, topk, device="cuda"), torch.empty(tokens, topk, device="cuda")
    ops.combine_backward(dout, y, rows, w, torch.empty_like(y), dw)
    want = (y.double()[rows.long()] * dout.double()[:, None]).sum(2)
    err = float((dw.double() / want - 1.0).abs().max())
    assert err <= (terms + 1) * U + width * 2.0 ** -52, err
