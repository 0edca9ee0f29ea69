"""The embedding of a vocabulary shard and its gradient on the GPU, against
tests/ops_reference.py.  Bounds (u = 2^-24): a looked-up element is one
product, u and half a step of its type; a gradient adds n rows one after
another: (n + 2) u of the sum of magnitudes and half a step of its type (with
`accumulate` one more addition)."""
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

    h = snac.snac_init(2)
    yield h
    snac.snac_finalize(h)


def host(t):
    return t.detach().double().cpu().numpy()


def matrix(torch, rows, width, dtype, g, shift=0, pad=0):
    wide = torch.full((rows + 1, shift + width + pad), 77.0, dtype=getattr(torch, DT[dtype]), device="cuda")
    m = wide[:rows, shift:shift + width]
    m.copy_(torch.from_numpy(g.normal(size=(rows, width)).astype(np.float32)))
    return wide, m


def untouched(wide, m, shift):
    rows, width = m.shape
    return bool((wide[rows:] == 77).all() and (wide[:, :shift] == 77).all() and (wide[:, shift + width:] == 77).all())


def far_ids(ids, id_type):
    """Some ids of no shard at all."""
    if ids.size > 6:
        ids[1], ids[2] = (2 ** 31 - 1, -(2 ** 31)) if id_type == "int32" else (2 ** 63 - 1, -(2 ** 63))
        ids[3] = -1
    return ids


# tokens, vocab, first, width, column shifts
SHAPES = [(1, 1, 0, 1, 0), (400, 50, 9, 8195, 1), (1, 50, 3, 2048, 0), (5, 7, 100, 9, 1), (64, 33, 0, 515, 3), (300, 1000, 0, 64, 0),
          (1000, 40, 20, 130, 2), (20, 300, 7, 8192, 0), (40, 64, 0, 2050, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("id_type", ["int32", "int64"])
@pytest.mark.parametrize("tokens,vocab,first,width,shift", SHAPES)
def test_embedding(torch, dtype, id_type, tokens, vocab, first, width, shift):
    g = np.random.default_rng(tokens * 3 + width)
    _, table = matrix(torch, vocab, width, dtype, g, shift, 2)
    wide, out = matrix(torch, tokens, width, dtype, g, shift, 1)
    ids = far_ids(g.integers(first - 5, first + vocab + 5, tokens), id_type)
    ops().embedding(table, torch.tensor(ids, dtype=getattr(torch, id_type), device="cuda"), out, first=first, scale=1.7)
    tab, got = host(table), host(out)
    for t, i in enumerate(int(v) for v in ids):
        want = tab[i - first] * np.float64(np.float32(1.7)) if first <= i < first + vocab else np.zeros(width)
        assert np.all(np.abs(got[t] - want) <= (U + ref.half_step(dtype)) * np.abs(want) * 1.01 + 1e-37), t
    assert untouched(wide, out, shift)


def test_embedding_of_batches_and_shards(torch):
    """[batch, length] ids; the shards' outputs add up to the whole table's, bit for bit."""
    g = np.random.default_rng(2)
    _, table = matrix(torch, 96, 200, "bf16", g)
    table = table.contiguous()
    ids = torch.tensor(g.integers(0, 96, (4, 31)), device="cuda")
    whole = torch.empty(4, 31, 200, dtype=torch.bfloat16, device="cuda")
    ops().embedding(table, ids, whole)
    assert torch.equal(whole, table[ids])
    parts = []
    for s in range(3):
        parts.append(torch.empty_like(whole))
        ops().embedding(table[32 * s:32 * (s + 1)], ids, parts[-1], first=32 * s)
    assert torch.equal(parts[0] + parts[1] + parts[2], whole)


def test_embedding_of_nothing(torch, handle):
    out = torch.full((3, 16), 5.0, device="cuda")
    ops().embedding(torch.empty(0, 16, device="cuda"), torch.arange(3, device="cuda"), out)
    assert (out == 0).all()
    ops().embedding(torch.ones(4, 16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), out[:0])
    dt = torch.full((9, 16), 5.0, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    ops().embedding_backward(out[:0], none, dt, handle, accumulate=True)
    assert (dt == 5).all()
    ops().embedding_backward(out[:0], none, dt, handle)
    assert (dt == 0).all()


def backward_case(torch, handle, dtype, grad, id_type, tokens, vocab, first, width, shift, accumulate, ids, pad=None):
    g = np.random.default_rng(tokens * 5 + width)
    _, d = matrix(torch, tokens, width, dtype, g, shift, 1)
    wide, dt = matrix(torch, vocab, width, grad, g, shift, 2)
    before = host(dt)
    ops().embedding_backward(d, torch.tensor(ids, dtype=getattr(torch, id_type), device="cuda"), dt, handle, first=first,
                             pad=pad, scale=0.75, accumulate=accumulate)
    want, mag, n = ref.embedding_backward(host(d), ids, first, vocab, pad, 0.75)
    got = host(dt)
    tol = (n + 2)[:, None] * U * mag
    if accumulate:
        same = n == 0
        assert np.array_equal(got[same], before[same])
        want = want + before
        tol = tol + U * (np.abs(want) + mag)
    tol = tol + ref.half_step(grad) * np.abs(want) * 1.01 + 1e-37
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)
    if not accumulate:
        assert np.all(got[n == 0] == 0)
    assert untouched(wide, dt, shift)


@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,vocab,first,width,shift", SHAPES)
def test_backward(torch, handle, dtype, grad, accumulate, tokens, vocab, first, width, shift):
    g = np.random.default_rng(tokens * 7 + width)
    id_type = "int64" if tokens % 2 else "int32"
    ids = far_ids(first - 3 + ((vocab + 6) * g.random(tokens) ** 3).astype(np.int64), id_type)
    backward_case(torch, handle, dtype, grad, id_type, tokens, vocab, first, width, shift, accumulate, ids,
                  pad=first + 1 if vocab > 2 else None)


@pytest.mark.parametrize("tokens", [7, 8, 9, 31, 32, 33, 65, 1000, 4096, 4097, 9000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_of_one_token(torch, handle, tokens, accumulate):
    """Every position the same token: one run over all chunks; one sort run and several."""
    backward_case(torch, handle, "f32", "f32", "int64", tokens, 5, 10, 70, 0, accumulate, np.full(tokens, 12))


@pytest.mark.parametrize("run", [1, 2, 31, 32, 33, 95])
@pytest.mark.parametrize("tokens", [700, 5000])
def test_backward_of_equal_runs(torch, handle, run, tokens):
    """Runs of one length, shuffled: their ends fall on, before and after the chunks' ends."""
    ids = np.random.default_rng(run).permutation(np.arange(tokens) // run)
    backward_case(torch, handle, "bf16", "f32", "int32", tokens, tokens // run + 2, 0, 40, 0, False, ids)


@pytest.mark.parametrize("vocab", [1023, 1024, 1025, 131072, 2 ** 20 - 1, 2 ** 20, 2 ** 20 + 5])
def test_backward_by_vocabulary(torch, handle, vocab):
    """One, two and three sort passes, and keys at the ends of their digits."""
    tokens, width = 9001, 16
    g = np.random.default_rng(vocab)
    ids = g.integers(0, vocab, tokens)
    ids[:500] = g.integers(max(0, vocab - 3), vocab, 500)
    ids[500:600] = vocab  # just past the end: another shard's
    d = torch.tensor(g.normal(size=(tokens, width)).astype(np.float32), device="cuda")
    dt = torch.full((vocab, width), 77.0, device="cuda")
    ops().embedding_backward(d, torch.tensor(ids, device="cuda"), dt, handle)
    keep = torch.tensor(np.flatnonzero(ids < vocab), device="cuda")
    at = torch.tensor(ids[ids < vocab], device="cuda")
    want = torch.zeros(vocab, width, dtype=torch.float64, device="cuda").index_add_(0, at, d[keep].double())
    mag = torch.zeros(vocab, width, dtype=torch.float64, device="cuda").index_add_(0, at, d[keep].double().abs())
    n = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    assert bool(((dt.double() - want).abs() <= (n[:, None] + 3) * U * mag).all())
    again = torch.empty_like(dt)
    ops().embedding_backward(d, torch.tensor(ids, device="cuda"), again, handle)
    assert torch.equal(again, dt), "not the same bits twice"


@pytest.mark.parametrize("width", [512, 515, 1030, 2047])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_of_ragged_widths(torch, handle, width, accumulate):
    """Widths whose last columns do not fill a wave; few tokens and many; every row and a few rows with tokens."""
    g = np.random.default_rng(width)
    for tokens, vocab in ((300, 40), (300, 900), (4500, 64)):
        ids = g.integers(-3, vocab + 3, tokens)
        backward_case(torch, handle, "bf16", "f32", "int64", tokens, vocab, 0, width, 0, accumulate, ids)


@pytest.mark.parametrize("dtype,grad,width", [("bf16", "f32", 4095), ("bf16", "f32", 4097), ("bf16", "bf16", 8200),
                                              ("f32", "f32", 12289), ("f32", "bf16", 16385)])
@pytest.mark.parametrize("tokens", [5, 200, 9000])
def test_backward_of_wide_rows(torch, handle, dtype, grad, width, tokens):
    """Rows whose zeros are more than one workgroup's; a few rows without a token, and most."""
    vocab = 9300 if tokens == 9000 else 230
    g = np.random.default_rng(width + tokens)
    ids = g.integers(0, vocab, tokens)
    d = torch.ones(tokens, width, dtype=getattr(torch, DT[dtype]), device="cuda")
    dt = torch.full((vocab, width + 3), 77.0, dtype=getattr(torch, DT[grad]), device="cuda")
    ops().embedding_backward(d, torch.tensor(ids, device="cuda"), dt[:, 1:width + 1], handle)
    n = torch.bincount(torch.tensor(ids, device="cuda"), minlength=vocab)  # small whole numbers: exact in bf16
    assert int(n.max()) <= 256
    assert torch.equal(dt[:, 1:width + 1], n[:, None].to(dt.dtype).expand(vocab, width))
    assert bool((dt[:, 0] == 77).all()) and bool((dt[:, width + 1:] == 77).all())


def test_offsets_past_32_bits(torch, handle):
    """A table and its gradient of more than 2^32 bytes: first and last rows, zeros between."""
    vocab, width = 150000, 8192
    ids = torch.tensor([0, vocab - 1, 131072, vocab - 1, 131071, vocab], device="cuda")
    table = torch.zeros(vocab, width, device="cuda")  # 4.9 GB
    rows = torch.randn(6, width, device="cuda")
    table[ids[:5]] = rows[[0, 3, 2, 3, 4]]
    out = torch.empty(6, width, device="cuda")
    ops().embedding(table, ids, out)
    assert torch.equal(out[:5], table[ids[:5]]) and (out[5] == 0).all()
    table.fill_(7.0)
    ops().embedding_backward(rows, ids, table, handle)
    assert torch.equal(table[0], rows[0]) and torch.equal(table[131072], rows[2]) and torch.equal(table[131071], rows[4])
    assert torch.equal(table[vocab - 1], rows[1] + rows[3])
    table[[0, 131071, 131072, vocab - 1]] = 0
    assert not bool(table.any())


@pytest.mark.parametrize("tokens", [0, 3, 9000])
def test_more_rows_than_a_launch_holds(torch, handle, tokens):
    """Zeros of 2^28 rows and some are 2^32 threads and some."""
    vocab = 2 ** 28 + 2 ** 24 + 5
    g = torch.Generator().manual_seed(tokens)
    ids = torch.randint(0, vocab, (tokens,), generator=g)
    ids[:3] = torch.tensor([vocab - 1, 2 ** 28, 0])[:tokens]
    ids = ids.cuda()
    table = torch.full((vocab, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    ops().embedding_backward(torch.ones(tokens, 1, device="cuda"), ids, table, handle)
    named, times = ids.unique(return_counts=True)
    assert torch.equal(table[named, 0].float(), times.float())
    table[named] = 0
    assert not bool(table.any())


def test_gradient_against_differences(torch, handle):
    """The lookup is linear in the table, so a difference of its outputs at two tables is exact but for rounding: each
    output is off by 2 half steps, over tokens of them, and the step divides it."""
    g = np.random.default_rng(4)
    vocab, width, tokens, h = 6, 10, 25, 0.5
    ids = torch.tensor(g.integers(0, vocab, tokens), device="cuda")
    table = torch.tensor(g.normal(size=(vocab, width)).astype(np.float32), device="cuda")
    d = torch.tensor(g.normal(size=(tokens, width)).astype(np.float32), device="cuda")
    dt = torch.empty_like(table)
    ops().embedding_backward(d, ids, dt, handle, scale=3.0)

    def value(t):
        out = torch.empty(tokens, width, device="cuda")
        ops().embedding(t, ids, out, scale=3.0)
        return (host(out) * host(d)).sum(), (np.abs(host(out)) * np.abs(host(d))).sum()

    for v, c in [(0, 0), (3, 9), (5, 4)]:
        up, down = table.clone(), table.clone()
        up[v, c] += h
        down[v, c] -= h
        (a, ma), (b, mb) = value(up), value(down)
        step = float(up[v, c].double() - down[v, c].double())
        assert abs((a - b) / step - float(dt[v, c])) <= 4 * U * (ma + mb) / step + (tokens + 2) * U * 3 * float(d.abs().sum())


def test_scratch(torch):
    import copy_reduce_snac_amd as snac

    tokens, vocab, width = 5000, 64, 512
    need = snac.snac_embedding_scratch(tokens, vocab, width)
    d = torch.ones(tokens, width, device="cuda")
    ids = torch.arange(tokens, device="cuda") % vocab
    dt = torch.empty(vocab, width, device="cuda")
    small = snac.snac_init(1, 8192)
    enough = snac.snac_init(1, -(-need // 4194304) * 4194304)
    try:
        with pytest.raises(snac.SnacError) as e:
            ops().embedding_backward(d, ids, dt, small)
        assert e.value.status == snac.SNAC_E_ARG and "scratch" in str(e.value)
        ops().embedding_backward(d, ids, dt, enough)
        want = torch.bincount(ids, minlength=vocab).float()
        assert torch.equal(dt, want[:, None].expand(vocab, width))
    finally:
        snac.snac_finalize(small)
        snac.snac_finalize(enough)
