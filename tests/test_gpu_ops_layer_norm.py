"""Layer norm and its gradients on the GPU, against tests/ops_step_reference.py.

Bounds, u = 2^-24, h = (x - mean) rstd, half = half a step of the output's type:
  out     x - near is off by u |d|, the mean of the d's by 7 u of their mean size
          (at most the deviation), x - mean by a rounding more; the squares' sum
          by 8 u and its root by half of that, rstd by a rounding more; two
          products and a sum of one rounding each:
          |w| u (10 |h| + 8) + u |out| + half |out|
  stats   mean: u |mean| + 8 u deviation; rstd: 8 u rstd
  dx      for the stats that the call got: h 2 u, g u, means of g 10 u and of
          g h 14 u of the terms' mean sizes (sums of a unit 7, rounding,
          1 / width, product), three operations more:
          u rstd (4 |g| + 14 mean|g| + 20 |h| mean|g h|) + half |dx|
  dweight 32 fused multiply-adds, 6 joinings of 64 rows side by side and a
          rounding, h 2: 41 u of the terms' sizes + half |dweight|; dbias likewise;
          accumulated ones with what was there among the sizes
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


def near(got, want, bound, what):
    got = host(got)
    assert got.shape == want.shape, what
    off = np.abs(got - want) - bound
    assert not np.isnan(got).any() and (off <= 0).all(), (what, np.unravel_index(np.argmax(off), off.shape), off.max())


def matrix(torch, values, dtype, shift=0, pad=0):
    """`values` in the columns shift .. of a wider matrix of canaries."""
    rows, width = values.shape
    wide = torch.full((rows + 1, shift + width + pad), 77.0, dtype=getattr(torch, DT[dtype]), device="cuda")
    m = wide[:rows, shift:shift + width]
    m.copy_(torch.from_numpy(np.asarray(values, np.float32)))
    return wide, m


def untouched(wide, m, shift):
    rows, width = m.shape
    return bool((wide[rows:] == 77).all() and (wide[:, :shift] == 77).all() and (wide[:, shift + width:] == 77).all())


def vector(torch, values, dtype, shift):
    return torch.from_numpy(np.concatenate([np.zeros(shift), values]).astype(np.float32)).to(getattr(torch, DT[dtype])).cuda()[shift:]


def out_bound(h, w, out, dtype):
    return np.abs(w) * U * (10 * np.abs(h) + 8) + (U + HALF[dtype]) * np.abs(out) + TINY


# every shape that is compiled, whole and not, and rows that go to the wide kernels
WIDTHS = [1, 2, 3, 7, 8, 63, 64, 65, 100, 128, 129, 250, 255, 256, 257, 511, 512, 513, 1000, 1024, 1030, 2047, 2048, 2049, 4096, 5003, 8192, 8200, 12001,
          16384, 16385, 30000, 33000]


@pytest.mark.parametrize("dtype,params", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("width", WIDTHS)
def test_both_ways(torch, ops, handle, dtype, params, width):
    g = np.random.default_rng(width)
    rows = 37 if width < 4000 else 9
    shift, pad = width % 3, width % 2
    xs = g.normal(size=(rows, width)) * np.exp(0.3 * g.normal(size=width)) + g.normal(size=width)
    wx, x = matrix(torch, xs, dtype, shift, pad)
    wide, out = matrix(torch, np.zeros((rows, width)), dtype, pad, shift)
    w = vector(torch, 1 + 0.2 * g.normal(size=width), params, shift)
    b = vector(torch, g.normal(size=width), params, pad)
    stats = torch.full((rows + 1, 2), 55.0, device="cuda")
    ops.layer_norm(x, w, b, out, eps=1e-5, stats=stats[:rows])
    torch.cuda.synchronize()
    assert untouched(wide, out, pad) and untouched(wx, x, shift) and (stats[rows:] == 55).all()
    hx, hw, hb = host(x), host(w), host(b)
    mean, rstd = ref.moments(hx, np.float32(1e-5))
    want = ref.layer_norm(hx, hw, hb, np.float32(1e-5))
    h = (hx - mean) * rstd
    near(out, want, out_bound(h, hw, np.abs(want) + np.abs(h * hw), dtype), "out")
    near(stats[:rows, :1], mean, U * np.abs(mean) + 8 * U / rstd, "mean")
    near(stats[:rows, 1:], rstd, 8 * U * rstd, "rstd")

    gs = g.normal(size=(rows, width))
    wg, dout = matrix(torch, gs, dtype, pad, shift)
    for accumulate, grad in ((False, "f32"), (True, "f32"), (False, "bf16"), (True, "bf16")):
        wide, dx = matrix(torch, np.zeros((rows, width)), dtype, shift, 1 + pad)
        dw, db = (torch.full((width + 2,), 3.0, dtype=getattr(torch, DT[grad]), device="cuda") for _ in "wb")
        ops.layer_norm_backward(dout, x, w, stats[:rows], dx, dw[1:-1], db[1:-1], handle, accumulate=accumulate)
        torch.cuda.synchronize()
        assert untouched(wide, dx, shift) and untouched(wg, dout, pad)
        assert all(float(v[0]) == 3 and float(v[-1]) == 3 for v in (dw, db))
        hs, hg = host(stats[:rows]), host(dout)
        want_dx, want_dw, want_db = ref.layer_norm_backward(hg, hx, hw, hs)
        h, up = (hx - hs[:, :1]) * hs[:, 1:], hg * hw
        mg, mgh = np.abs(up).mean(axis=1, keepdims=True), np.abs(up * h).mean(axis=1, keepdims=True)
        near(dx, want_dx, U * hs[:, 1:] * (4 * np.abs(up) + 14 * mg + 20 * np.abs(h) * mgh) + HALF[dtype] * np.abs(want_dx) + TINY, "dx")
        old = 3.0 if accumulate else 0.0
        for got, sums, size in ((dw, want_dw, np.abs(hg * h).sum(axis=0)), (db, want_db, np.abs(hg).sum(axis=0))):
            near(got[1:-1], sums + old, 41 * U * (size + old) + HALF[grad] * np.abs(sums + old), (grad, accumulate))


@pytest.mark.parametrize("tokens", [1, 2, 31, 4096, 4097, 16500, 40001])
@pytest.mark.parametrize("dtype,width", [("bf16", 40), ("bf16", 200), ("f32", 260), ("bf16", 2050)])
def test_many_tokens(torch, ops, handle, dtype, width, tokens):
    """Sums over many tokens are not off by more than over few; whole numbers come out whole."""
    if tokens * width > 1 << 25:
        tokens //= 2
    dt = getattr(torch, DT[dtype])
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    # stats of mean 0 and rstd 1: h is x, and x and dout are small whole numbers
    x = torch.randint(-2, 3, (tokens, width), generator=g, device="cuda").to(dt)
    dout = torch.randint(-2, 3, (tokens, width), generator=g, device="cuda").to(dt)
    stats = torch.tensor([0.0, 1.0], device="cuda").repeat(tokens, 1)
    dx = torch.empty_like(x)
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    ops.layer_norm_backward(dout, x, None, stats, dx, dw, db, handle)
    assert torch.equal(dw.double(), (x.double() * dout.double()).sum(0))
    assert torch.equal(db.double(), dout.double().sum(0))
    # one column at a time: the other is left alone
    only = torch.empty(width, device="cuda")
    ops.layer_norm_backward(dout, x, None, stats, dx, only, None, handle)
    assert torch.equal(only, dw)
    only.zero_()
    ops.layer_norm_backward(dout, x, None, stats, dx, None, only, handle)
    assert torch.equal(only, db)
    again = torch.empty_like(dx)
    ops.layer_norm_backward(dout, x, None, stats, again, None, None)  # no context
    assert torch.equal(again, dx)


@pytest.mark.parametrize("dtype,width,tokens", [("f32", 4100, 8193), ("bf16", 8300, 16400), ("f32", 9000, 3700), ("bf16", 20001, 3300)])
def test_more_tokens_than_turns(torch, ops, handle, dtype, width, tokens):
    """More than 32 turns of the workgroups that fill the chip, held rows and wide ones: whole numbers come out whole."""
    dt = getattr(torch, DT[dtype])
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    x = torch.randint(-2, 3, (tokens, width), generator=g, device="cuda", dtype=torch.int8).to(dt)
    dout = torch.randint(-2, 3, (tokens, width), generator=g, device="cuda", dtype=torch.int8).to(dt)
    stats = torch.tensor([0.0, 1.0], device="cuda").repeat(tokens, 1)
    dx = torch.empty_like(x)
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    ops.layer_norm_backward(dout, x, None, stats, dx, dw, db, handle)
    assert torch.equal(dw, (x * dout).sum(0, dtype=torch.float32)) and torch.equal(db, dout.sum(0, dtype=torch.float32))
    for t in (0, tokens // 2, tokens - 1):
        one = torch.empty_like(dx[:1])
        ops.layer_norm_backward(dout[t:t + 1], x[t:t + 1], None, stats[t:t + 1], one, None, None, handle)
        assert torch.equal(one[0], dx[t]), t


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [300, 5000, 40000])
def test_in_place_and_without_parameters(torch, ops, handle, dtype, width):
    g = np.random.default_rng(7)
    x = torch.from_numpy(g.normal(size=(50, width)).astype(np.float32)).to(getattr(torch, DT[dtype])).cuda()
    w = torch.from_numpy(g.normal(size=width).astype(np.float32)).cuda()
    stats, dout = torch.empty(50, 2, device="cuda"), torch.randn(50, width, device="cuda").to(x.dtype)
    for weight, bias in ((None, None), (w, None), (None, w), (w, w)):
        out = torch.empty_like(x)
        ops.layer_norm(x, weight, bias, out, stats=stats)
        hx, hw = host(x), None if weight is None else host(weight)
        want = ref.layer_norm(hx, hw, None if bias is None else host(bias), np.float32(1e-5))
        mean, rstd = ref.moments(hx, np.float32(1e-5))
        h = (hx - mean) * rstd
        hw = np.ones(width) if hw is None else hw
        near(out, want, out_bound(h, hw, np.abs(want) + np.abs(h * hw), dtype), (weight is None, bias is None))
        same = x.clone()
        ops.layer_norm(same, weight, bias, same)
        assert torch.equal(same, out)
        dx, dw = torch.empty_like(x), torch.empty(width, device="cuda")
        ops.layer_norm_backward(dout, x, weight, stats, dx, dw, None, handle)
        same, dw2 = dout.clone(), torch.empty_like(dw)
        ops.layer_norm_backward(same, x, weight, stats, same, dw2, None, handle)
        assert torch.equal(same, dx) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [3, 27, 131, 300, 505, 1999, 5003, 9999, 25001])
def test_rows_with_a_part_of_a_unit(torch, ops, handle, dtype, width):
    """The shared end of a row: in place, over the rows of a workgroup, as if each row came alone."""
    rows = min(20001, (1 << 23) // width)
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    x, dout = (torch.randn(rows, width, generator=g, device="cuda").to(getattr(torch, DT[dtype])) for _ in "xd")
    w, b = torch.randn(2, width, generator=g, device="cuda")
    out, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, 2, device="cuda")
    dw, db = torch.empty(2, width, device="cuda")
    ops.layer_norm(x, w, b, out, stats=stats)
    ops.layer_norm_backward(dout, x, w, stats, dx, dw, db, handle)
    same = x.clone()
    ops.layer_norm(same, w, b, same)
    assert torch.equal(same, out)
    same, dw2, db2 = dout.clone(), torch.empty_like(dw), torch.empty_like(db)
    ops.layer_norm_backward(same, x, w, stats, same, dw2, db2, handle)
    assert torch.equal(same, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    for t in (0, 1, rows // 2, rows - 2, rows - 1):
        one = torch.empty_like(x[:1])
        ops.layer_norm(x[t:t + 1], w, b, one)
        assert torch.equal(one[0], out[t]), t
        ops.layer_norm_backward(dout[t:t + 1], x[t:t + 1], w, stats[t:t + 1], one, None, None, handle)
        assert torch.equal(one[0], dx[t]), t
    h = (x.double() - stats[:, :1].double()) * stats[:, 1:].double()
    hg = dout.double()
    # as dweight above: a workgroup's turns are at most 32 for any number of tokens
    for got, terms in ((dw, hg * h), (db, hg)):
        assert ((got.double() - terms.sum(0)).abs() <= 41 * U * terms.abs().sum(0) + TINY).all()


@pytest.mark.parametrize("width", [5, 640, 3000, 9001, 40000])
def test_rows_far_from_zero(torch, ops, width):
    """A constant row is 0 with any eps, and a row far from 0 is as good as the same row near it."""
    x = torch.full((6, width), 1000.123, device="cuda")
    x[1] = -3.0e7
    x[2] = 0.1
    out, stats = torch.empty_like(x), torch.empty(6, 2, device="cuda")
    ops.layer_norm(x, None, None, out, eps=1e-12, stats=stats)
    assert torch.equal(out, torch.zeros_like(out)) and torch.equal(stats[:, 0], x[:, 0])
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    small = torch.randint(-50, 51, (6, width), generator=g, device="cuda").float()
    ops.layer_norm(small + 1048576.0, None, None, out, stats=stats)  # these sums are exact
    hx = host(small)
    mean, rstd = ref.moments(hx, np.float32(1e-5))
    h = (hx - mean) * rstd
    near(out, h, out_bound(h, 1.0, np.abs(h), "f32"), "far")
    near(stats[:, 1:], rstd, 8 * U * rstd, "rstd")


def test_values_that_are_not_finite(torch, ops, handle):
    """NaN and infinity stay in their rows; the sums over tokens get them."""
    x = torch.randn(8, 700, device="cuda")
    clean = torch.empty_like(x)
    ops.layer_norm(x, None, None, clean)
    bad = x.clone()
    bad[2, 5], bad[4, 699], bad[6, 0] = float("nan"), float("inf"), -float("inf")
    out, stats = torch.empty_like(x), torch.empty(8, 2, device="cuda")
    ops.layer_norm(bad, None, None, out, stats=stats)
    for r in range(8):
        assert bool(out[r].isnan().all()) if r in (2, 4, 6) else torch.equal(out[r], clean[r])
    flat = torch.ones(1, 9, device="cuda")
    ops.layer_norm(flat, None, None, flat, eps=0.0)
    assert bool(flat.isnan().all())
    dx, dw, db = torch.empty_like(x), torch.empty(700, device="cuda"), torch.empty(700, device="cuda")
    ops.layer_norm(x, None, None, out, stats=stats)
    dout = torch.randn_like(x)
    dout[3, 17] = float("nan")
    ops.layer_norm_backward(dout, x, None, stats, dx, dw, db, handle)
    assert bool(dx[3].isnan().all()) and not dx[[0, 1, 2, 4, 5, 6, 7]].isnan().any()
    assert dw.isnan().nonzero().flatten().tolist() == db.isnan().nonzero().flatten().tolist() == [17]


def test_no_tokens(torch, ops, handle):
    x, st = torch.empty(0, 24, device="cuda"), torch.empty(0, 2, device="cuda")
    dw, db = torch.full((24,), 4.0, device="cuda"), torch.full((24,), 4.0, device="cuda")
    ops.layer_norm(x, dw, None, x, stats=st)
    ops.layer_norm_backward(x, x, None, st, x, dw, db, handle, accumulate=True)
    assert bool((dw == 4).all() and (db == 4).all())
    ops.layer_norm_backward(x, x, None, st, x, dw, db, handle)
    assert bool((dw == 0).all() and (db == 0).all())


def test_too_little_scratch(torch, ops):
    import copy_reduce_snac_amd as snac

    h = snac.snac_init(1, 8192)
    try:
        x, st = torch.randn(600, 4096, device="cuda"), torch.zeros(600, 2, device="cuda")
        dw = torch.empty(4096, device="cuda")
        assert snac.snac_layer_norm_scratch(600, 4096, "f32") > 8192
        with pytest.raises(snac.SnacError, match="scratch"):
            ops.layer_norm_backward(x, x, None, st, torch.empty_like(x), dw, None, h)
    finally:
        snac.snac_finalize(h)
