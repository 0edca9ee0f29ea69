"""The global gradient norm and clipping on the GPU, against NumPy in
binary64.  Bounds (u = 2^-24): the norm is summed in binary64 and rounded once
(its own error is below n 2^-53), 1.01 u; the factor adds 1e-6 and divides
(2 u) by it; the product rounds to binary32 and to the type: 5 u and half a
step."""
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


def host(t):
    return t.detach().double().cpu().numpy()


LISTS = [
    [(1, "f32", 0)], [(1, "bf16", 1)], [(7, "bf16", 3)], [(0, "f32", 0), (5, "f32", 1), (0, "bf16", 0)],
    [(4096, "f32", 0), (8192, "bf16", 0)], [(4097, "f32", 1), (8193, "bf16", 5), (3, "f32", 2)],
    [(100003, "bf16", 7), (33, "f32", 3), (65536, "f32", 0), (1, "bf16", 0), (250001, "f32", 2)],
    [(i * 37 % 400 + 1, "f32" if i % 3 else "bf16", i % 5) for i in range(700)],
    [(3_000_001, "bf16", 1), (2_000_003, "f32", 3)],
]


def tensors(torch, spec, g, scale=1.0):
    """Tensors at element offsets in buffers of canaries."""
    bufs, ts = [], []
    for n, dtype, off in spec:
        b = torch.full((n + off + 3,), 77.0, dtype=getattr(torch, DT[dtype]), device="cuda")
        b[off:off + n] = torch.from_numpy((g.normal(size=n) * scale).astype(np.float32)).cuda()
        bufs.append(b)
        ts.append(b[off:off + n])
    return bufs, ts


@pytest.mark.parametrize("which", range(len(LISTS)))
@pytest.mark.parametrize("where", ["in place", "apart"])
@pytest.mark.parametrize("clips", [True, False])
def test_norm_and_clip(torch, which, where, clips):
    spec = LISTS[which]
    g = np.random.default_rng(which)
    bufs, ts = tensors(torch, spec, g)
    xs = [host(t) for t in ts]
    obufs, outs = (bufs, ts) if where == "in place" else tensors(torch, [(n, d, (o + 1) % 8) for n, d, o in spec], g)
    lst = ops().GradList(ts, None if where == "in place" else outs)
    want = np.sqrt(sum((x ** 2).sum() for x in xs))
    max_norm = float(np.float32(want * (0.3 if clips else 2.0)))
    norm = torch.full((3,), 55.0, device="cuda")
    ops().clip_grad_norm(lst, max_norm, norm[1:2])
    got = float(norm[1])
    assert abs(got - want) <= 1.01 * U * want
    assert norm[0] == 55 and norm[2] == 55
    factor = min(1.0, max_norm / (want + 1e-6))
    for (n, dtype, off), x, out, b, o in zip(spec, xs, outs, obufs, range(len(spec))):
        y = host(out)
        if factor == 1.0:
            assert np.array_equal(y, x)
        else:
            assert np.all(np.abs(y - x * factor) <= (5 * U + ref.half_step(dtype)) * np.abs(x * factor) * 1.01 + 1e-37)
        lo = off if where == "in place" else (off + 1) % 8
        assert bool((b[:lo] == 77).all()) and bool((b[lo + n:] == 77).all()), "written outside"
    if where == "apart":
        assert all(np.array_equal(host(t), x) for t, x in zip(ts, xs)), "a source was written"
    lst.close()


@pytest.mark.parametrize("where", ["in place", "apart"])
def test_large_list(torch, where):
    """Enough tiles for the counters that hand them out (128 MiB on 256 CUs), three calls in a row: whole outputs, in
    binary64 on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    sizes = [(50_000_003, torch.bfloat16, 3), (17, torch.float32, 1), (40_000_001, torch.float32, 5),
             (9_000_000, torch.bfloat16, 0)]
    bufs = [torch.empty(n + 16, dtype=d, device="cuda").normal_(generator=g) for n, d, _ in sizes]
    ts = [b[o:o + n] for b, (n, _, o) in zip(bufs, sizes)]
    obufs = bufs if where == "in place" else [torch.full_like(b, 77.0) for b in bufs]
    outs = ts if where == "in place" else [b[o + 1:o + 1 + n] for b, (n, _, o) in zip(obufs, sizes)]
    lst = ops().GradList(ts, None if where == "in place" else outs)
    norm = torch.empty(1, device="cuda")
    for _ in range(3):
        xs = [t.clone() for t in ts]
        want = float(sum(x.double().square().sum() for x in xs)) ** 0.5
        max_norm = float(np.float32(want / 2))
        ops().clip_grad_norm(lst, max_norm, norm)
        assert abs(float(norm) - want) <= 1.01 * U * want
        for x, y in zip(xs, outs):
            e = x.double() * (max_norm / (want + 1e-6))
            half = ref.half_step("bf16" if x.dtype == torch.bfloat16 else "f32")
            assert bool(((y.double() - e).abs() <= (5 * U + half) * e.abs() * 1.01 + 1e-37).all())
        if where == "apart":
            assert all(torch.equal(t, x) for t, x in zip(ts, xs))
            assert all(bool((b[:o + 1] == 77).all()) and bool((b[o + 1 + n:] == 77).all())
                       for b, (n, _, o) in zip(obufs, sizes))


def test_empty_list(torch):
    norm = torch.full((1,), 9.0, device="cuda")
    for ts in ([], [torch.empty(0, device="cuda")]):
        norm.fill_(9.0)
        lst = ops().GradList(ts)
        ops().clip_grad_norm(lst, 1.0, norm)
        assert float(norm) == 0.0


def test_no_overflow_or_underflow(torch):
    """Squares past binary32's range on both sides."""
    norm = torch.empty(1, device="cuda")
    for v, n in [(1e30, 16), (1e-30, 1024), (3e38, 1), (2.0 ** -126, 4)]:
        x = torch.full((n,), v, device="cuda")
        ops().grad_norm(ops().GradList([x]), norm)
        want = float(x[0].double()) * np.sqrt(n)
        assert abs(float(norm) - want) <= 1.01 * U * want, v
    ops().grad_norm(ops().GradList([torch.full((16,), 3e38, device="cuda")]), norm)
    assert float(norm) == float("inf")  # 1.2e39 is past binary32


@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_what_is_not_finite(torch, bad):
    """As the formula has it: an infinite norm gives zeros and NaN where the infinities were, a NaN all NaN."""
    x = torch.ones(1000, device="cuda")
    x[123] = float(bad)
    y = torch.ones(50, dtype=torch.bfloat16, device="cuda")
    norm = torch.empty(1, device="cuda")
    ops().clip_grad_norm(ops().GradList([x, y]), 1.0, norm)
    if bad == "nan":
        assert torch.isnan(norm).all() and torch.isnan(x).all() and torch.isnan(y).all()
    else:
        assert float(norm) == float("inf")
        assert torch.isnan(x[123]) and int((x == 0).sum()) == 999 and (y == 0).all()


def test_again_and_again(torch):
    """A list is read anew at each call, and its sums have one order: the same bits each time."""
    g = np.random.default_rng(6)
    _, ts = tensors(torch, [(700_001, "f32", 1), (300_000, "bf16", 2)], g)
    lst = ops().GradList(ts)
    norm = torch.empty(40, device="cuda")
    for i in range(20):
        ops().grad_norm(lst, norm[i:i + 1])
    ts[0].mul_(2.0)
    for i in range(20, 40):
        ops().grad_norm(lst, norm[i:i + 1])
    got = norm.cpu()
    assert (got[:20] == got[0]).all() and (got[20:] == got[20]).all() and got[0] != got[20]


def test_in_one_call_and_in_two(torch):
    """snac_clip_grad_norm is snac_grad_norm, then snac_clip_grads: the same bits."""
    g = np.random.default_rng(7)
    for spec in LISTS:
        _, ts = tensors(torch, spec, g)
        outs = [[torch.empty_like(t) for t in ts] for _ in range(2)]
        norm = torch.empty(2, device="cuda")
        ops().clip_grad_norm(ops().GradList(ts, outs[0]), 0.5, norm[:1])
        two = ops().GradList(ts, outs[1])
        ops().grad_norm(two, norm[1:])
        ops().clip_grads(two, norm[1:], 0.5)
        assert norm[0] == norm[1]
        assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_max_norm_of_zero(torch):
    x = torch.ones(100, device="cuda")
    norm = torch.empty(1, device="cuda")
    ops().clip_grad_norm(ops().GradList([x]), 0.0, norm)
    assert (x == 0).all() and float(norm) == 10.0


def test_closed_list(torch):
    lst = ops().GradList([torch.ones(4, device="cuda")])
    lst.close()
    with pytest.raises(ValueError):
        ops().grad_norm(lst, torch.empty(1, device="cuda"))
