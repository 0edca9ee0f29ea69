"""Layer norm's gradient of rows whose mean times 1 / deviation or whose sums pass
binary32's range, and rows that do not vary, or hardly.

Bounds as in test_gpu_ops_layer_norm.py (u = 2^-24, h = (x - mean) rstd):
  dx      u rstd (4 |g| + 14 mean|g| + 20 |h| mean|g h|) + half |dx|
  dweight 41 u of the terms' sizes + half |dweight|; dbias likewise
"""
from __future__ import annotations

import numpy as np
import pytest

import ops_step_reference as ref
from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24
DT = {"f32": "float32", "bf16": "bfloat16"}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 1e-37


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


def host(t):
    return t.detach().double().cpu().numpy()


# rows of less than a unit, and rows that fill a part of every shape
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [1, 3, 5, 7, 9, 32, 100, 130, 300, 1000, 1027, 3000, 5000, 5003, 9000, 17000, 20001])
def test_gradient_of_large_rows(torch, ops, handle, dtype, width):
    rows = 40
    g = np.random.default_rng(width)
    x = torch.from_numpy(g.normal(size=(rows, width)).astype(np.float32)).to(getattr(torch, DT[dtype])).cuda()
    stats = np.concatenate(ref.moments(host(x), 1e-5), axis=1)
    for r, (size, rstd) in enumerate([(2.0 ** 121, 1e-5 ** -0.5), (-2.0 ** 121, 1e-5 ** -0.5), (2.0 ** 64, 2.0 ** 70)]):
        x[r] = size  # constant rows
        stats[r] = size, rstd
    stats = torch.from_numpy(stats.astype(np.float32)).cuda()
    dout = torch.from_numpy(g.normal(size=(rows, width)).astype(np.float32)).to(x.dtype).cuda()
    w = torch.from_numpy((1 + 0.2 * g.normal(size=width)).astype(np.float32)).cuda()
    dx, dw, db = torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    ops.layer_norm_backward(dout, x, w, stats, dx, dw, db, handle)
    hx, hg, hw, hs = host(x), host(dout), host(w), host(stats)
    want_dx, want_dw, want_db = ref.layer_norm_backward(hg, hx, hw, hs)
    h, up = (hx - hs[:, :1]) * hs[:, 1:], hg * hw
    mg, mgh = np.abs(up).mean(axis=1, keepdims=True), np.abs(up * h).mean(axis=1, keepdims=True)
    bound = U * hs[:, 1:] * (4 * np.abs(up) + 14 * mg + 20 * np.abs(h) * mgh) + HALF[dtype] * np.abs(want_dx) + TINY
    got = host(dx)
    assert not np.isnan(got).any(), np.isnan(got).any(axis=1).nonzero()
    assert (np.abs(got - want_dx) <= bound).all()
    for got, sums, size in ((dw, want_dw, np.abs(hg * h).sum(axis=0)), (db, want_db, np.abs(hg).sum(axis=0))):
        assert (np.abs(host(got) - sums) <= 41 * U * size + U * np.abs(sums) + TINY).all()


# widths whose reciprocal is exact or rounded down or up, in the shapes that hold a row and the wide one
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [1, 3, 49, 64, 237, 479, 1000, 1700, 1871, 3001, 5003, 7101, 7798, 13001, 33001, 41003])
def test_constant_rows_without_eps(torch, ops, dtype, width):
    """0 over 0: NaN whatever the constant, as the formula has it; with the smallest eps 0."""
    g = np.random.default_rng(width)
    values = (g.normal(size=64) * 10.0 ** g.uniform(-3, 5, size=64)).astype(np.float32)
    x = torch.from_numpy(values).to(getattr(torch, DT[dtype])).cuda().unsqueeze(1).repeat(1, width)
    out, stats = torch.empty_like(x), torch.empty(64, 2, device="cuda")
    ops.layer_norm(x, None, None, out, eps=0.0, stats=stats)
    assert bool(out.isnan().all()), out.isnan().all(dim=1).logical_not().nonzero().flatten().tolist()
    assert torch.equal(stats[:, 0], x[:, 0].float())
    ops.layer_norm(x, None, None, out, eps=2.0 ** -149, stats=stats)
    assert bool((out == 0).all()) and torch.equal(stats[:, 0], x[:, 0].float())


@pytest.mark.parametrize("width", [60, 130, 700, 1671, 2927, 4532, 5990, 16001, 40001])
def test_rows_that_hardly_vary(torch, ops, width):
    """Rows far from 0 that differ by a unit in the last place here and there, as good as any row near 0: distances from
    a binary32 number near the mean are exact there, so the bound of test_gpu_ops_layer_norm.py stays
    u (10 |h| + 8) + 2 u |out|, however far that number is from the mean in deviations."""
    g = np.random.default_rng(width)
    x = np.repeat((g.uniform(1, 2, size=(50, 1)) * 2.0 ** 24).astype(np.float32), width, axis=1)
    for row in x:
        at = g.integers(0, width, g.integers(1, max(2, width // 50)))
        row[at] = np.nextafter(row[at], np.float32(np.inf))
    t = torch.from_numpy(x).cuda()
    out, stats = torch.empty_like(t), torch.empty(50, 2, device="cuda")
    ops.layer_norm(t, None, None, out, stats=stats)
    mean, rstd = ref.moments(x, np.float32(1e-5))
    h = (x.astype(np.float64) - mean) * rstd
    assert (np.abs(host(out) - h) <= U * (12 * np.abs(h) + 8) + TINY).all(), (np.abs(host(out) - h) / (U * (12 * np.abs(h) + 8))).max()
    assert (np.abs(host(stats[:, :1]) - mean) <= U * np.abs(mean) + 8 * U / rstd).all()
    assert (np.abs(host(stats[:, 1:]) - rstd) <= 8 * U * rstd).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [5000, 5003, 8192, 9000, 16001, 20001])
def test_gradient_of_large_gradients(torch, ops, handle, dtype, width):
    """Sums of a row that pass binary32's range, of terms and with means far below it."""
    rows = 20
    g = np.random.default_rng(width)
    x = torch.from_numpy(g.normal(size=(rows, width)).astype(np.float32)).to(getattr(torch, DT[dtype])).cuda()
    stats = torch.from_numpy(np.concatenate(ref.moments(host(x), 1e-5), axis=1).astype(np.float32)).cuda()
    dout = torch.full_like(x, 2.0 ** 116)  # sum g passes it
    dout[::2] = dout[::2] * torch.where(x[::2] > 0, 1.0, -1.0)  # sum g h does, sum g does not
    dx = torch.empty_like(x)
    ops.layer_norm_backward(dout, x, None, stats, dx, None, None, handle)
    hx, hg, hs = host(x), host(dout), host(stats)
    want, _, _ = ref.layer_norm_backward(hg, hx, None, hs)
    h = (hx - hs[:, :1]) * hs[:, 1:]
    mg, mgh = np.abs(hg).mean(axis=1, keepdims=True), np.abs(hg * h).mean(axis=1, keepdims=True)
    bound = U * hs[:, 1:] * (4 * np.abs(hg) + 14 * mg + 20 * np.abs(h) * mgh) + HALF[dtype] * np.abs(want)
    got = host(dx)
    assert np.isfinite(got).all() and (np.abs(got - want) <= bound).all()
