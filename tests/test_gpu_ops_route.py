"""Routing to experts and its gradient on the GPU, against the binary64
definition (tests/ops_reference.py).

Choices have to be equal.  Bounds (u = 2^-24): a weight is an exponential of
a difference of logits (its rounding and the exponential's own: |d| + 2 half
steps, |d| up to 30 here), over a sum of up to 1024 such terms added 16 a lane
and then over 6 levels (22 half steps), two more for the quotient and the
scale: 30 + 2 + 22 + (30 + 2) + 2 < 96 u of the weight.  A gradient is such a
product with a difference of sums of 32 terms: 128 u of score * (|a| + sum
|r a|), and half a step of its type."""
from __future__ import annotations

import numpy as np
import pytest

import ops_reference as ref
from gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24


def ops():
    from copy_reduce_snac_amd import operators

    return operators


def torch_():
    import torch

    return torch


DT = {"f32": "float32", "bf16": "bfloat16"}


def device(x, dtype, pad=0):
    """x as a device matrix of the type, with `pad` canary columns after each row."""
    torch = torch_()
    t = torch.full((x.shape[0], x.shape[1] + pad), 77.0, dtype=getattr(torch, DT[dtype]), device="cuda")
    t[:, :x.shape[1]] = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    return t[:, :x.shape[1]]


def host(t):
    return t.detach().double().cpu().numpy()


def run(x, topk, dtype, pad=0, bias=None, **kw):
    torch = torch_()
    lx = device(x, dtype, pad)
    w = torch.full((x.shape[0] + 1, topk), 55.0, device="cuda")
    ids = torch.full((x.shape[0] + 1, topk), 55, dtype=torch.int32, device="cuda")
    b = None if bias is None else torch.tensor(np.asarray(bias, np.float32), device="cuda")
    ops().route(lx, w[:-1], ids[:-1], bias=b, **kw)
    torch.cuda.synchronize()
    assert (w[-1] == 55).all() and (ids[-1] == 55).all(), "written past the end"
    return host(lx), host(w[:-1]), ids[:-1].cpu().numpy()


def check(x, topk, dtype, pad=0, bias=None, **kw):
    xs, w, ids = run(x, topk, dtype, pad, bias, **kw)
    b = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    for t in range(xs.shape[0]):
        rw, rid = ref.route(xs[t], topk, bias=b, **kw)
        assert ids[t].tolist() == rid.tolist(), f"row {t}"
        assert np.all(np.abs(w[t] - rw) <= 96 * U * np.abs(rw) + 1e-37), f"row {t}: {w[t]} {rw}"


CONFIGS = [
    dict(n=8, topk=2), dict(n=60, topk=4, renorm=False), dict(n=64, topk=6), dict(n=65, topk=1),
    dict(n=1, topk=1), dict(n=1024, topk=32, renorm=False), dict(n=513, topk=8, scale=2.5),
    dict(n=256, topk=8, groups=8, topk_groups=4), dict(n=256, topk=8, groups=8, topk_groups=4, group_top=1),
    dict(n=160, topk=6, groups=8, topk_groups=3), dict(n=72, topk=3, groups=4, topk_groups=1),
    dict(n=64, topk=4, groups=64, topk_groups=8), dict(n=12, topk=12, groups=3, topk_groups=3),
    dict(n=320, topk=10, groups=5, topk_groups=2),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_route(dtype, score, biased, cfg):
    cfg = dict(cfg)
    n, topk = cfg.pop("n"), cfg.pop("topk")
    g = np.random.default_rng(n * 7 + topk)
    x = g.normal(size=(37, n)) * 2
    x[3] = -np.inf                                    # nothing to choose
    x[4, : n - 1] = -np.inf                           # one expert left
    x[5] = 0.25                                       # all equal
    x[6] = np.finfo(np.float32).min if dtype == "f32" else -3.3895313892515355e38  # the type's lowest value
    x[7, ::2] = -np.inf
    x[8] = -90.0 + g.normal(size=n)                   # sigmoids near the end of binary32
    x[9] *= 8
    bias = g.normal(size=n) * 0.05 if biased else None
    check(x, topk, dtype, pad=0 if n % 2 else 5, bias=bias, score=score, **cfg)


@pytest.mark.parametrize("tokens", [0, 1, 3, 5000])
def test_token_counts(tokens):
    g = np.random.default_rng(tokens)
    x = g.normal(size=(tokens, 96))
    xs, w, ids = run(x, 4, "f32", score="sigmoid")
    for t in range(0, tokens, 97):
        rw, rid = ref.route(xs[t], 4, score="sigmoid")
        assert ids[t].tolist() == rid.tolist()
        assert np.all(np.abs(w[t] - rw) <= 96 * U * np.abs(rw))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("copies", [1, 1200])
def test_keys_one_step_apart(score, groups, copies):
    """Logits one binary32 step apart, whose scores agree in binary32, and biases that do not part them; few of them
    and all, so that the choice is in doubt at its end, inside it and between groups; one token a wave and several."""
    n = 64
    g = np.random.default_rng(3)
    base = np.float32(2.0)
    steps = g.permutation(n)
    x = np.stack([np.float32(base) + steps.astype(np.float32) * np.float32(2.0 ** -22),
                  np.float32(base) - steps.astype(np.float32) * np.float32(2.0 ** -22)])
    far = g.normal(size=(40, n)) - 3
    for row in far:  # pairs and threes
        at = g.permutation(n)[:12].reshape(6, 2)
        for i, (p, q) in enumerate(at):
            row[p] = 3 - 0.4 * i
            row[q] = np.float32(row[p]) + np.float32(2.0 ** -22) * g.integers(-1, 2)
    x = np.concatenate([x, far]).astype(np.float32)
    kw = dict(score=score, groups=groups, topk_groups=max(1, groups // 2))
    for bias in (None, np.zeros(n), np.full(n, 0.125)):
        check(x, 8, "f32", bias=bias, **kw)
        if copies > 1:
            _, w1, ids1 = run(x, 8, "f32", bias=bias, **kw)
            _, w, ids = run(np.tile(x, (copies // 20, 1)), 8, "f32", bias=bias, **kw)
            assert (ids.reshape(-1, *ids1.shape) == ids1).all()
            assert np.abs(w.reshape(-1, *w1.shape) - w1).max() <= 192 * U


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("cfg", [c for c in CONFIGS if c["topk"] <= 8] + [
    dict(n=10, topk=8), dict(n=16, topk=12), dict(n=60, topk=9), dict(n=292, topk=10, groups=4, topk_groups=2),
    dict(n=256, topk=12, renorm=False), dict(n=500, topk=8, groups=5, topk_groups=3), dict(n=96, topk=5, groups=48, topk_groups=7),
    dict(n=1020, topk=7, groups=3, topk_groups=2), dict(n=900, topk=3, groups=30, topk_groups=4)],
    ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_many_tokens(dtype, score, biased, cfg):
    """Several tokens a wave; coarse logits (ties), fine ones, masked experts; every row's choice, in NumPy at once."""
    cfg = dict(cfg)
    n, topk = cfg.pop("n"), cfg.pop("topk")
    g = np.random.default_rng(n * 11 + topk)
    tokens = 4099
    x = g.normal(size=(tokens, n)) * 2
    x[::3] = np.round(x[::3] * 16) / 16
    x[::7, g.random(n) < 0.2] = -np.inf
    x[5] = -np.inf
    bias = g.normal(size=n) * 0.05 if biased else None
    xs, w, ids = run(x, topk, dtype, bias=bias, score=score, **cfg)
    b = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    with np.errstate(all="ignore"):
        m = xs.max(axis=1, keepdims=True)
        s = 1 / (1 + np.exp(-xs)) if score == "sigmoid" else np.exp(xs - m) / np.exp(xs - m).sum(axis=1, keepdims=True)
    key = np.where(xs == -np.inf, -np.inf, s if b is None else s + b)
    gr = cfg.get("groups", 1)
    if gr > 1:
        k3 = np.sort(key.reshape(tokens, gr, n // gr), axis=2)[:, :, ::-1]
        worth = k3[:, :, 0] + k3[:, :, 1] if cfg.get("group_top", 2) == 2 and n // gr > 1 else k3[:, :, 0]
        best = np.argsort(-worth, axis=1, kind="stable")[:, :cfg["topk_groups"]]
        ok = np.zeros((tokens, gr), bool)
        np.put_along_axis(ok, best, np.take_along_axis(worth, best, 1) > -np.inf, 1)
        key = np.where(np.repeat(ok, n // gr, axis=1), key, -np.inf)
    want = np.argsort(-key, axis=1, kind="stable")[:, :topk]
    want = np.where(np.take_along_axis(key, want, 1) == -np.inf, -1, want)
    bad = np.flatnonzero((ids != want).any(axis=1))
    assert bad.size == 0, f"rows {bad[:5]}: {ids[bad[:3]]} {want[bad[:3]]}"
    for t in range(0, tokens, 41):
        rw, _ = ref.route(xs[t], topk, bias=b, score=score, **cfg)
        assert np.all(np.abs(w[t] - rw) <= 96 * U * np.abs(rw) + 1e-37), t


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_past_32_bits(dtype):
    """Rows 2^30 elements apart, forward and backward."""
    torch = torch_()
    n, step = 96, 2 ** 30
    buf = torch.zeros(2 * step + n, dtype=getattr(torch, DT[dtype]), device="cuda")
    x = buf.as_strided((3, n), (step, 1))
    x.copy_(torch.randn(3, n, device="cuda"))
    near = x.contiguous()
    got = []
    for lx in (x, near):
        w, ids = torch.empty(3, 5, device="cuda"), torch.empty(3, 5, dtype=torch.int32, device="cuda")
        ops().route(lx, w, ids, score="sigmoid")
        dx = torch.empty_like(near)
        ops().route_backward(lx, ids, w, dx, score="softmax", renorm=False)
        got.append((w, ids, dx))
    ops().route_backward(near, got[1][1], got[1][0], x, score="softmax", renorm=False)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(x, got[1][2])
    x.zero_()
    assert not bool(buf.any())


def test_more_tokens_than_a_launch_holds():
    """2^28 tokens and some are 2^32 threads and some: the same as calls of 2^26 tokens."""
    torch = torch_()
    n, part = 2 ** 28 + 77, 2 ** 26
    x = torch.empty(n, 16, dtype=torch.bfloat16, device="cuda").normal_()
    w, ids = torch.empty(n, 1, device="cuda"), torch.empty(n, 1, dtype=torch.int32, device="cuda")
    dx = torch.empty_like(x)
    ops().route(x, w, ids, renorm=False)
    ops().route_backward(x, ids, w, dx, renorm=False)
    for lo in range(0, n, part):
        px = x[lo:lo + part]
        pw, pids, pdx = torch.full_like(w[:len(px)], -1), torch.full_like(ids[:len(px)], -1), torch.empty_like(px)
        ops().route(px, pw, pids, renorm=False)
        ops().route_backward(px, pids, pw, pdx, renorm=False)
        # the last part is small enough for another shape, whose softmax adds up in another order
        same = len(px) == part
        assert torch.equal(ids[lo:lo + part], pids), lo
        assert torch.equal(w[lo:lo + part], pw) if same else torch.allclose(w[lo:lo + part], pw, rtol=192 * U, atol=0), lo
        assert torch.equal(dx[lo:lo + part], pdx) if same else bool(dx[lo:].isfinite().all()), lo


def test_ties_go_to_the_lowest_index():
    g = np.random.default_rng(9)
    x = g.integers(-2, 3, size=(200, 128)).astype(np.float64) / 4
    for kw in (dict(score="softmax"), dict(score="sigmoid", bias=np.zeros(128)),
               dict(score="sigmoid", groups=8, topk_groups=3, bias=g.integers(0, 2, 128) / 8)):
        check(x, 9, "bf16", **kw)


@pytest.mark.parametrize("tokens", [6, 3000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_equal_in_binary64(tokens, score):
    """Different logits whose binary64 scores saturate or underflow: equal keys, the lower index first."""
    g = np.random.default_rng(13)
    x = g.normal(size=(6, 64)) * 20
    x[0] += 60
    x[1] -= 800
    x[2, 5:] -= 1500
    x[3] = 18 + g.normal(size=64) * 3
    x[4, 1:] = 1e-20 * g.random(63)
    check(np.resize(x, (6, 64)), 7, "f32", score=score)
    for top in (1, 2):  # and groups by their largest keys, or by two
        y = np.tile(x, (tokens // 6, 1))
        _, _, ids = run(y, 4, "f32", score=score, groups=8, topk_groups=2, group_top=top)
        for t in range(6):
            want = ref.route(host(device(x, "f32"))[t], 4, score=score, groups=8, topk_groups=2, group_top=top)[1]
            assert (ids.reshape(-1, 6, 4)[:, t] == want).all(), (top, t)
    xs, w, ids = run(np.tile(x, (tokens // 6, 1)), 7, "f32", score=score)
    assert (ids.reshape(-1, 6, 7) == ids[:6]).all()


def test_signed_zeros_are_equal():
    x = np.zeros((2, 70))
    x[0, ::3] = -0.0
    x[1, 1::2] = -0.0
    check(x, 5, "f32", score="softmax")
    check(x, 5, "f32", score="sigmoid")


def test_masked_by_the_bias():
    g = np.random.default_rng(11)
    x = g.normal(size=(6, 32))
    bias = g.normal(size=32) * 0.1
    bias[::2] = -np.inf
    check(x, 20, "f32", bias=bias, score="sigmoid")


def test_nan_and_infinity():
    x = np.random.default_rng(12).normal(size=(4, 40))
    x[0, 7] = np.nan
    x[1, 9] = np.inf
    x[2, 30] = np.nan
    x[2, 31] = -np.inf
    for score in ("softmax", "sigmoid"):
        xs, w, ids = run(x, 3, "f32", score=score, renorm=False)
        for t in range(4):
            rw, rid = ref.route(xs[t], 3, score, renorm=False)
            assert ids[t].tolist() == rid.tolist(), (score, t)
            assert np.array_equal(np.isnan(w[t]), np.isnan(rw)), (score, t)
            ok = ~np.isnan(rw)
            assert np.all(np.abs(w[t] - rw)[ok] <= 96 * U * np.abs(rw)[ok])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("n,topk", [(8, 2), (60, 4), (64, 8), (129, 3), (256, 8), (513, 5), (1024, 32)])
def test_route_backward(dtype, score, renorm, n, topk):
    torch = torch_()
    g = np.random.default_rng(n + topk)
    tokens = 23
    x = g.normal(size=(tokens, n)) * 2
    x[2, ::3] = -np.inf
    x[3] = -np.inf
    x[4] = -80.0 + g.normal(size=n)
    lx = device(x, dtype, 3)
    ids = np.stack([g.permutation(n)[:topk] for _ in range(tokens)]).astype(np.int32)
    ids[2] = [i if i % 3 else -1 for i in ids[2]]
    ids[3] = -1
    ids[5, -1] = -1
    ids[6, 0] = n        # out of range: no part in it
    ids[7, 0] = -(2 ** 31)
    dw = g.normal(size=(tokens, topk)).astype(np.float32)
    wide = torch.full((tokens + 1, n + 2), 77.0, dtype=lx.dtype, device="cuda")
    dx = wide[:tokens, 1:n + 1]
    ops().route_backward(lx, torch.tensor(ids, device="cuda"), torch.tensor(dw, device="cuda"), dx, score=score,
                         renorm=renorm, scale=2.5)
    torch.cuda.synchronize()
    assert (wide[-1] == 77).all() and (wide[:, 0] == 77).all() and (wide[:, -1] == 77).all(), "written outside"
    xs, got = host(lx), host(dx)
    for t in range(tokens):
        want = ref.route_backward(xs[t], ids[t], dw[t], score, renorm, 2.5)
        s = ref.scores(xs[t], score)
        ok = [(int(i), 2.5 * abs(float(d))) for i, d in zip(ids[t], dw[t]) if 0 <= i < n]
        size = np.zeros(n)
        if ok:
            at, a = np.array([i for i, _ in ok]), np.array([d for _, d in ok])
            r = ref.chosen_scores(xs[t], s, at, score, renorm)
            if score == "softmax" and not renorm:
                size[at] = a
                size = s * (size + np.dot(r, a))
            else:
                size[at] = r * (a + (np.dot(r, a) if renorm else 0))
        tol = 128 * U * size + ref.half_step(dtype) * np.abs(want) * 1.01 + 1e-37
        assert np.all(np.abs(got[t] - want) <= tol), (t, np.max(np.abs(got[t] - want) - tol))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    """The kernel's gradient against central differences of the binary64 forward: off by h^2 / 6 times a third
    derivative (below 100 here), and by 128 half steps of terms below 10."""
    torch = torch_()
    g = np.random.default_rng(21)
    x = g.normal(size=(1, 19)).astype(np.float32).astype(np.float64)
    ids = np.array([[4, 11, 0]], np.int32)
    dw = g.normal(size=(1, 3)).astype(np.float32)
    dx = torch.empty(1, 19, device="cuda")
    ops().route_backward(device(x, "f32"), torch.tensor(ids, device="cuda"), torch.tensor(dw, device="cuda"), dx,
                         score=score, renorm=renorm, scale=1.5)
    got = host(dx)[0]
    h = 1e-4
    for j in range(19):
        up, down = x[0].copy(), x[0].copy()
        up[j] += h
        down[j] -= h
        d = np.dot(dw[0], ref.weights_of(up, ids[0], score, renorm, 1.5) - ref.weights_of(down, ids[0], score, renorm, 1.5)) / (2 * h)
        assert abs(d - got[j]) <= h * h / 6 * 100 + 128 * U * 10
