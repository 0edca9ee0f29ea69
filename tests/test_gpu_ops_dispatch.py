"""The dispatch plan, dispatch, combine and combine's gradient on the GPU,
against tests/ops_reference.py.  The plan and dispatch are exact.  Bounds
(u = 2^-24): a combined element is topk fused multiply-adds, topk u of the sum
of magnitudes, and half a step of its type; dy is one product rounded once or
twice; dweights adds width / 64 products a lane and 6 levels over the lanes:
(width / 64 + 16) u of the sum of magnitudes (a lane takes whole units, up to 8
elements more than its share)."""
from __future__ import annotations

import numpy as np
import pytest

import ops_reference as ref
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

    h = snac.snac_init(1)
    yield h
    snac.snac_finalize(h)


def host(t):
    return t.detach().double().cpu().numpy()


def matrix(torch, rows, width, dtype, g, shift=0, pad=0):
    """A random matrix in the columns shift .. shift + width of a wider one of canaries."""
    wide = torch.full((rows + 1, shift + width + pad), 77.0, dtype=getattr(torch, DT[dtype]), device="cuda")
    m = wide[:rows, shift:shift + width]
    m.copy_(torch.from_numpy(g.normal(size=(rows, width)).astype(np.float32)))
    return wide, m


def untouched(wide, m, shift):
    rows, width = m.shape
    return bool((wide[rows:] == 77).all() and (wide[:, :shift] == 77).all() and (wide[:, shift + width:] == 77).all())


@pytest.mark.parametrize("id_type", ["int32", "int64"])
@pytest.mark.parametrize("slots,experts", [(0, 5), (1, 1), (7, 3), (64, 8), (1000, 60), (8192, 256), (8193, 256),
                                           (12289, 1024), (70001, 12), (262144, 128), (1500000, 1000)])
def test_plan(torch, handle, id_type, slots, experts):
    g = np.random.default_rng(slots + experts)
    ids = (experts * g.random(slots) ** 2).astype(np.int64)
    if slots > 5:
        ids[g.random(slots) < 0.1] = -1
        ids[3], ids[4] = experts, (2 ** 31 - 1 if id_type == "int32" else 2 ** 40)
        ids[5] = -(2 ** 31) if id_type == "int32" else -(2 ** 63)
    t = torch.tensor(ids, dtype=getattr(torch, id_type), device="cuda")
    counts = torch.full((experts + 1,), 55, dtype=torch.int32, device="cuda")
    row = torch.full((slots + 1,), 55, dtype=torch.int32, device="cuda")
    back = torch.full((slots + 1,), 55, dtype=torch.int32, device="cuda")
    for _ in range(2):  # the scratch of one call does not matter to the next
        ops().dispatch_plan(t, counts[:-1], row[:-1], back[:-1], handle)
    torch.cuda.synchronize()
    assert counts[-1] == 55 and row[-1] == 55 and back[-1] == 55, "written past the end"
    order = np.argsort(np.where((ids >= 0) & (ids < experts), ids, experts), kind="stable")
    n = int(((ids >= 0) & (ids < experts)).sum())
    want_row = np.full(slots, -1)
    want_row[order[:n]] = np.arange(n)
    want_back = np.full(slots, -1)
    want_back[:n] = order[:n]
    assert np.array_equal(counts[:-1].cpu().numpy(), np.bincount(ids[(ids >= 0) & (ids < experts)], minlength=experts))
    assert np.array_equal(row[:-1].cpu().numpy(), want_row)
    assert np.array_equal(back[:-1].cpu().numpy(), want_back)


@pytest.mark.parametrize("value", [0, 6, -1])
def test_plan_of_one_expert(torch, handle, value):
    """Every slot to one expert, or to none."""
    n, experts = 50000, 7
    t = torch.full((n,), value, dtype=torch.int32, device="cuda")
    counts = torch.empty(experts, dtype=torch.int32, device="cuda")
    row, back = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    ops().dispatch_plan(t, counts, row, back, handle)
    want = torch.arange(n, dtype=torch.int32, device="cuda") if value >= 0 else torch.full_like(row, -1)
    assert torch.equal(row, want) and torch.equal(back, want)
    assert counts.tolist() == [n if e == value else 0 for e in range(experts)]


def test_plan_without_room(torch):
    import copy_reduce_snac_amd as snac

    h = snac.snac_init(1, 8192)
    try:
        n, experts = 100000, 1024
        i = torch.zeros(n, dtype=torch.int32, device="cuda")
        c = torch.zeros(experts, dtype=torch.int32, device="cuda")
        with pytest.raises(snac.SnacError) as e:
            ops().dispatch_plan(i, c, torch.empty_like(i), torch.empty_like(i), h)
        assert e.value.status == snac.SNAC_E_ARG and "scratch" in str(e.value)
    finally:
        snac.snac_finalize(h)


# tokens, topk, width, column shifts of x and out, columns after them
SHAPES = [(1, 1, 1, 0, 0), (300, 3, 8195, 1, 2), (1, 8, 2048, 0, 0), (3, 2, 7, 1, 2), (5, 3, 8, 0, 8), (33, 4, 515, 3, 2), (17, 8, 1030, 0, 2),
          (9, 32, 64, 0, 0), (40, 2, 2049, 1, 0), (6, 1, 8192, 0, 0), (2000, 4, 100, 0, 4), (11, 5, 4097, 2, 1)]


def slots_of(g, tokens, k, rows):
    """Distinct rows for the slots that are not dropped; one token loses all."""
    m = tokens * k
    r = np.full(m, -1)
    keep = g.random(m) > 0.15
    if m > 4:
        keep[:k] = False
    r[keep] = g.permutation(rows)[:keep.sum()]
    if m > 8:  # out of range: dropped as well
        r[m - 1] = rows
        r[m - 2] = -(2 ** 31)
    return r.reshape(tokens, k).astype(np.int32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,topk,width,shift,pad", SHAPES)
def test_dispatch(torch, dtype, tokens, topk, width, shift, pad):
    g = np.random.default_rng(tokens * 31 + width)
    rows = tokens * topk + 3
    r = slots_of(g, tokens, topk, rows)
    _, x = matrix(torch, tokens, width, dtype, g, shift, pad)
    wide, out = matrix(torch, rows, width, dtype, g, pad, shift)
    want = host(out)
    ops().dispatch(x, torch.tensor(r, device="cuda"), out)
    xs = host(x)
    for t in range(tokens):
        for k in range(topk):
            if 0 <= r[t, k] < rows:
                want[r[t, k]] = xs[t]
    assert np.array_equal(host(out), want)
    assert untouched(wide, out, pad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,topk,width,shift,pad", SHAPES)
def test_combine(torch, dtype, weighted, tokens, topk, width, shift, pad):
    g = np.random.default_rng(tokens * 37 + width)
    rows = tokens * topk + 3
    r = slots_of(g, tokens, topk, rows)
    _, y = matrix(torch, rows, width, dtype, g, shift, pad)
    wide, out = matrix(torch, tokens, width, dtype, g, pad, shift)
    w = g.normal(size=(tokens, topk)).astype(np.float32)
    w[(r < 0) | (r >= rows)] = np.nan  # not looked at
    wt = torch.tensor(w, device="cuda") if weighted else None
    ops().combine(y, torch.tensor(r, device="cuda"), wt, out)
    want, mag = ref.combine(host(y), r, w.astype(np.float64) if weighted else None)
    got = host(out)
    tol = topk * U * mag + ref.half_step(dtype) * np.abs(want) * 1.01 + 1e-37
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)
    assert untouched(wide, out, pad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tokens,topk,width,shift,pad", SHAPES)
def test_combine_backward(torch, dtype, in_place, tokens, topk, width, shift, pad):
    g = np.random.default_rng(tokens * 41 + width)
    rows = tokens * topk + 3
    r = slots_of(g, tokens, topk, rows)
    _, d = matrix(torch, tokens, width, dtype, g, pad, shift)
    wide_y, y = matrix(torch, rows, width, dtype, g, shift, pad)
    wide, dy = (wide_y, y) if in_place else matrix(torch, rows, width, dtype, g, pad, shift)
    w = g.normal(size=(tokens, topk)).astype(np.float32)
    ds, ys, want = host(d), host(y), host(dy)
    dw = torch.full((tokens + 1, topk), 55.0, device="cuda")
    ops().combine_backward(d, y, torch.tensor(r, device="cuda"), torch.tensor(w, device="cuda"), dy, dw[:-1])
    got, gw = host(dy), host(dw[:-1])
    assert (dw[-1] == 55).all()
    for t in range(tokens):
        for k in range(topk):
            if 0 <= r[t, k] < rows:
                want[r[t, k]] = float(w[t, k]) * ds[t]
                p = ds[t] * ys[r[t, k]]
                assert abs(gw[t, k] - p.sum()) <= (width / 64 + 16) * U * np.abs(p).sum() + 1e-37
            else:
                assert gw[t, k] == 0
    tol = (U + ref.half_step(dtype)) * np.abs(want) * 1.01 + 1e-37
    assert np.all(np.abs(got - want) <= tol)
    assert untouched(wide, dy, shift if in_place else pad)


def test_combine_is_the_gradient_of_dispatch(torch):
    """<dispatch(x), g> = <x, combine(g)>, both sides in binary64 of the kernels' outputs: dispatch is exact, combine's
    rounding is (topk + 1) half steps of the sum of magnitudes."""
    g = np.random.default_rng(8)
    tokens, topk, width = 50, 3, 130
    r = slots_of(g, tokens, topk, tokens * topk)
    _, x = matrix(torch, tokens, width, "f32", g)
    _, gr = matrix(torch, tokens * topk, width, "f32", g)
    out = torch.zeros(tokens * topk, width, device="cuda")
    back = torch.empty(tokens, width, device="cuda")
    rt = torch.tensor(r, device="cuda")
    ops().dispatch(x, rt, out)
    ops().combine(gr, rt, None, back)
    a, b = (host(out) * host(gr)).sum(), (host(x) * host(back)).sum()
    assert abs(a - b) <= (topk + 1) * U * (np.abs(host(out)) * np.abs(host(gr))).sum()


def test_rows_past_32_bits(torch):
    """A packed buffer of more than 2^32 bytes: the last rows, and nothing around them."""
    width, rows = 8192, 270000  # 4.4 GB of bf16
    out = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(4, width, device="cuda").bfloat16()
    r = torch.tensor([[rows - 1, 5], [262143, 262144], [rows - 2, -1], [0, 131072]], dtype=torch.int32, device="cuda")
    ops().dispatch(x, r, out)
    for t, k, row in [(0, 0, rows - 1), (0, 1, 5), (1, 0, 262143), (1, 1, 262144), (2, 0, rows - 2), (3, 0, 0), (3, 1, 131072)]:
        assert torch.equal(out[row], x[t])
    assert int((out != 0).any(dim=1).sum()) == 7
    back = torch.empty(4, width, dtype=torch.bfloat16, device="cuda")
    ops().combine(out, r, None, back)
    assert torch.equal(back, torch.cat([x[:2] * 2, x[2:3], x[3:] * 2]))
