"""Layer norm, the balance loss and distillation on the CPU: every refusal of
the C ABI, which must come before anything touches a GPU, and those of the
tensor-level calls."""
from __future__ import annotations

import ctypes

import pytest

import copy_reduce_snac_amd as snac

E = snac.SNAC_E_ARG
A, B, C, D, F, G, H = (0x100000 * i for i in range(1, 8))
FAR = 1 << 45


def refused(fn, *args, says: str = "") -> None:
    with pytest.raises(snac.SnacError) as e:
        fn(*args)
    assert e.value.status == E, str(e.value)
    assert says in str(e.value), str(e.value)


def test_layer_norm():
    def f(x=A, ld=32, w=B, b=C, pt="f32", t=8, n=32, eps=1e-5, dt="bf16", out=D, ld_out=32, stats=F):
        return (snac.snac_layer_norm, x, ld, w, b, pt, t, n, eps, dt, out, ld_out, stats)

    refused(*f(dt="u32"), says="dtype")
    refused(*f(pt="byte"), says="param_dtype")
    for eps in (-1e-9, float("nan"), float("inf")):
        refused(*f(eps=eps), says="eps")
    refused(*f(ld=31), says="stride")
    refused(*f(ld_out=31), says="stride")
    refused(*f(x=0), says="x is NULL")
    refused(*f(out=0), says="out is NULL")
    refused(*f(w=B + 2), says="weight not aligned")
    refused(*f(b=C + 1), says="bias not aligned")
    refused(*f(x=A + 1), says="x not aligned")
    refused(*f(stats=F + 2), says="stats not aligned")
    refused(*f(out=A + 64), says="overlaps")
    refused(*f(out=A, ld_out=33), says="overlaps")  # x, but with other rows
    refused(*f(out=B), says="overlaps")
    refused(*f(stats=C), says="overlaps")
    refused(*f(stats=D), says="overlaps")
    refused(*f(n=1 << 31, ld=1 << 31, ld_out=1 << 31), says="width")
    refused(*f(t=snac.SNAC_MAX_BYTES // 64 + 1, out=FAR, stats=2 * FAR), says="SNAC_MAX_BYTES")
    refused(*f(t=(1 << 64) - 1), says="SNAC_MAX_BYTES")
    snac.snac_layer_norm(0, 32, 0, 0, "f32", 0, 32, 1e-5, "f32", 0, 32)  # nothing to do
    snac.snac_layer_norm(0, 0, 0, 0, "f32", 4, 0, 1e-5, "f32", 0, 0, 0)


def test_layer_norm_backward():
    def f(g=A, ld_g=32, x=B, ld=32, w=C, pt="f32", stats=D, t=8, n=32, dt="bf16", dx=F, ld_dx=32, dw=G, db=H, gt="f32", acc=0):
        return (snac.snac_layer_norm_backward, None, g, ld_g, x, ld, w, pt, stats, t, n, dt, dx, ld_dx, dw, db, gt, acc)

    refused(*f(dt="byte"), says="dtype")
    refused(*f(pt="u32"), says="param_dtype")
    refused(*f(gt="u32"), says="grad_dtype")
    refused(*f(acc=2), says="accumulate")
    for kw in ({"ld": 31}, {"ld_g": 31}, {"ld_dx": 31}):
        refused(*f(**kw), says="stride")
    for kw, name in (({"g": 0}, "dout"), ({"x": 0}, "x"), ({"stats": 0}, "stats"), ({"dx": 0}, "dx")):
        refused(*f(**kw), says=f"{name} is NULL")
    refused(*f(dx=B), says="overlaps")
    refused(*f(dx=A, ld_dx=33), says="overlaps")  # dout, but with other rows
    refused(*f(dx=A + 64), says="overlaps")
    refused(*f(dx=D), says="overlaps")
    refused(*f(dw=C), says="overlaps")
    refused(*f(db=G), says="overlaps")
    refused(*f(db=G + 64), says="overlaps")
    refused(*f(dw=G + 2), says="aligned")
    refused(*f(stats=D + 1), says="aligned")
    refused(*f(), says="ctx")  # the sums over tokens need scratch
    refused(*f(dx=A), says="ctx")  # in place is right
    refused(*f(dw=0), says="ctx")
    refused(*f(n=1, ld=1, ld_g=1, ld_dx=1, t=1 << 34, g=FAR, x=2 * FAR, stats=3 * FAR, dx=4 * FAR, w=0), says="tokens")
    n = 20000  # rows too wide for a workgroup's registers need scratch for their sums too
    refused(*f(ld=n, ld_g=n, ld_dx=n, n=n, dw=0, db=0), says="ctx")
    snac.snac_layer_norm_backward(None, 0, 32, 0, 32, 0, "f32", 0, 0, 32, "f32", 0, 32, 0, 0, "f32")
    snac.snac_layer_norm_backward(None, 0, 0, 0, 0, 0, "f32", 0, 4, 0, "f32", 0, 0, G, H, "f32")
    s = snac.snac_layer_norm_scratch
    assert s(0, 32, "f32") == s(8, 0, "f32") == s(8, 1 << 31, "f32") == s(8, 32, "u32") == 0
    assert s(1 << 34, 1, "f32") == 0
    assert s(1, 32, "f32") >= 2 * 32 * 4
    assert s(1 << 20, 4096, "bf16") <= (1 << 20) * 4096 // 4  # an eighth of the rows


def test_balance():
    r = snac.router(16, 4)

    def f(rt=r, x=A, ld=16, ids=B, t=8, dt="f32", load=C):
        return (snac.snac_balance_load, None, rt, x, ld, ids, t, dt, load)

    for rt, says in [(snac.router(0, 1), "experts"), (snac.router(1025, 1), "experts"), (snac.router(16, 0), "topk"),
                     (snac.router(16, 17), "topk"), (snac.router(64, 33), "topk"), (snac.router(16, 4, 2), "score")]:
        refused(*f(rt=rt), says=says)
    refused(*f(rt=None), says="router")
    refused(*f(dt="u32"), says="dtype")
    refused(*f(ld=15), says="stride")
    refused(*f(x=0), says="logits")
    refused(*f(ids=0), says="ids")
    refused(*f(load=0), says="load")
    refused(*f(load=B), says="overlaps")
    refused(*f(load=A + 64), says="overlaps")
    refused(*f(load=C + 2), says="aligned")
    refused(*f(t=snac.SNAC_MAX_IDS // 4 + 1, ids=FAR, load=2 * FAR), says="SNAC_MAX_IDS")
    refused(*f(t=(1 << 64) - 1), says="SNAC_MAX_BYTES")
    refused(*f(), says="ctx")

    refused(snac.snac_balance_loss, A, 0, 1.0, B, says="experts")
    refused(snac.snac_balance_loss, A, 1025, 1.0, B, says="experts")
    refused(snac.snac_balance_loss, 0, 16, 1.0, B, says="load")
    refused(snac.snac_balance_loss, A, 16, 1.0, 0, says="loss")
    refused(snac.snac_balance_loss, A, 16, 1.0, A + 4, says="overlaps")

    def b(rt=r, x=A, ld=16, ids=B, load=C, dloss=D, t=8, dt="f32", dx=F, ld_d=16, acc=0):
        return (snac.snac_balance_backward, rt, x, ld, ids, load, 1.0, dloss, t, dt, dx, ld_d, acc)

    refused(*b(rt=snac.router(16, 17)), says="topk")
    refused(*b(dt="byte"), says="dtype")
    refused(*b(acc=-1), says="accumulate")
    refused(*b(ld=15), says="stride")
    refused(*b(ld_d=15), says="stride")
    for kw, name in (({"x": 0}, "logits"), ({"ids": 0}, "ids"), ({"load": 0}, "load"), ({"dx": 0}, "dlogits")):
        refused(*b(**kw), says=f"{name} is NULL")
    for at in (A, B, C, D):
        refused(*b(dx=at), says="overlaps")
    refused(*b(dloss=D + 1), says="aligned")
    snac.snac_balance_backward(r, 0, 16, 0, 0, 1.0, None, 0, "f32", 0, 16)


def teacher(ids=A, size=8, t=B, dt="f32", k=4, vocab=64, tau=2.0):
    return snac.teacher(ids, size, t, dt, k, vocab, tau)


BAD = [(teacher(size=2), "id_bytes"), (teacher(dt="u32"), "dtype"), (teacher(k=0), "topk"), (teacher(k=257), "topk"),
       (teacher(tau=0.0), "temperature"), (teacher(tau=-1.0), "temperature"), (teacher(tau=float("nan")), "temperature"),
       (teacher(tau=1e-30), "temperature"), (teacher(tau=float("inf")), "temperature"), (teacher(vocab=0), "vocab"),
       (teacher(vocab=-1), "vocab"), (teacher(vocab=snac.SNAC_MAX_BYTES + 1), "vocab"), (None, "teacher")]


def test_distill():
    assert ctypes.sizeof(snac.snac_teacher) == 40

    def f(h=None, z=C, ld=64, t=8, dt="bf16", loss=D, stats=F):
        return (snac.snac_distill, h or teacher(), z, ld, t, dt, loss, stats)

    def s(h=None, z=C, ld=16, first=32, n=16, t=8, dt="bf16", part=D):
        return (snac.snac_distill_shard, h or teacher(), z, ld, first, n, t, dt, part)

    def j(h=None, parts=C, n=4, t=8, loss=D, stats=F):
        return (snac.snac_distill_join, h or teacher(), parts, n, t, loss, stats)

    def b(h=None, z=C, ld=16, first=32, n=16, stats=D, dloss=F, t=8, dt="bf16", dz=G, ld_d=16):
        return (snac.snac_distill_backward, h or teacher(), z, ld, first, n, stats, dloss, 1.0, t, dt, dz, ld_d)

    for h, says in BAD:
        refused(snac.snac_distill, h, C, 64, 8, "f32", D, F, says=says)
        refused(snac.snac_distill_shard, h, C, 64, 0, 1, 8, "f32", D, says=says)
        refused(snac.snac_distill_join, h, C, 1, 8, D, F, says=says)
        refused(snac.snac_distill_backward, h, C, 64, 0, 1, D, None, 1.0, 8, "f32", G, 64, says=says)
    for make in (f, s, b):
        refused(*make(dt="u32"), says="dtype")
        refused(*make(z=0), says="logits is NULL")
        refused(*make(z=C + 1), says="aligned")
        refused(*make(ld=15), says="stride")
        refused(*make(t=(1 << 64) - 1), says="SNAC_MAX_BYTES")
    for make in (f, s, j, b):
        refused(*make(h=teacher(ids=0)), says="ids is NULL")
        refused(*make(h=teacher(ids=A + 4)), says="ids not aligned")
        refused(*make(h=teacher(t=0)), says="logits is NULL")
        refused(*make(h=teacher(t=B + 2)), says="logits not aligned")
        refused(*make(h=teacher(ids=D)), says="overlaps") if make is not b else refused(*make(dz=A), says="overlaps")
    for make in (s, b):
        for first, n in ((-1, 4), (65, 0), (60, 5), (0, 65), (1 << 62, 1)):
            refused(*make(first=first, n=n, ld=80), says="columns")
    refused(snac.snac_distill, teacher(vocab=1 << 31), C, 1 << 31, 8, "bf16", D, F, says="width")
    refused(*f(ld=63), says="stride")
    refused(*f(loss=0), says="loss")
    refused(*f(stats=0), says="stats")
    refused(*f(stats=D), says="overlaps")
    refused(*f(loss=C), says="overlaps")
    refused(*s(part=0), says="part")
    refused(*s(part=C), says="overlaps")
    refused(*j(n=0), says="shards")
    refused(*j(n=17), says="shards")
    refused(*j(parts=0), says="parts")
    refused(*j(loss=C), says="overlaps")
    refused(*b(dz=0), says="dlogits is NULL")
    refused(*b(dz=C, ld_d=17), says="overlaps")  # logits, but with other rows
    refused(*b(dz=C + 32), says="overlaps")
    refused(*b(dz=D), says="overlaps")
    refused(*b(ld_d=15), says="stride")
    refused(*b(stats=0), says="stats")
    # nothing to do
    snac.snac_distill(teacher(ids=0, t=0), 0, 64, 0, "f32", 0, 0)
    snac.snac_distill_shard(teacher(ids=0, t=0), 0, 64, 0, 64, 0, "f32", 0)
    snac.snac_distill_join(teacher(ids=0, t=0), 0, 4, 0, 0, 0)
    snac.snac_distill_backward(teacher(ids=0, t=0), 0, 64, 0, 64, 0, None, 1.0, 0, "f32", 0, 64)
    snac.snac_distill_backward(teacher(), 0, 0, 64, 0, 0, None, 1.0, 8, "f32", 0, 0)


def test_tensor_level():
    """The tensor-level calls look at shapes, types and strides before devices."""
    import torch

    from copy_reduce_snac_amd import operators as ops

    x = torch.zeros(4, 16)
    w, st = torch.ones(16), torch.zeros(4, 2)
    with pytest.raises(TypeError):
        ops.layer_norm(x.double(), w, w, x.double())
    with pytest.raises(TypeError):
        ops.layer_norm(x, w, w, x.bfloat16())
    with pytest.raises(TypeError):
        ops.layer_norm(x, w, w.bfloat16(), x)
    with pytest.raises(ValueError):
        ops.layer_norm(x, w[:15], None, x)
    with pytest.raises(ValueError):
        ops.layer_norm(x, None, None, torch.zeros(4, 15))
    with pytest.raises(ValueError):
        ops.layer_norm(x, torch.ones(32)[::2], None, x)
    with pytest.raises(ValueError):
        ops.layer_norm(x, w, w, x, stats=torch.zeros(4))
    with pytest.raises(ValueError, match="current device"):
        ops.layer_norm(x, w, w, x, stats=st)  # right in all but the device
    with pytest.raises(TypeError):
        ops.layer_norm_backward(x, x, w, st, x, w, w.bfloat16())
    with pytest.raises(ValueError):
        ops.layer_norm_backward(x, x[:3], w, st, x, w, None)
    with pytest.raises(ValueError, match="current device"):
        ops.layer_norm_backward(x, x, w, st, x, w, w)

    ids, load = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(2, 16)
    with pytest.raises(TypeError):
        ops.balance_load(x, ids.long(), load, 1)
    with pytest.raises(ValueError):
        ops.balance_load(x, ids, load[:, :15], 1)
    with pytest.raises(KeyError):
        snac.router(16, 2, "tanh")
    with pytest.raises(ValueError):
        ops.balance_loss(load[0], st[0, :1])
    with pytest.raises(ValueError):
        ops.balance_loss(load, st)
    with pytest.raises(ValueError):
        ops.balance_backward(x, ids, load, x[:, :15])
    with pytest.raises(ValueError):
        ops.balance_backward(x, ids, load, x.clone(), dloss=st)
    with pytest.raises(ValueError, match="current device"):
        ops.balance_backward(x, ids, load, x.clone())

    t, loss = torch.zeros(4, 2), torch.zeros(4)
    with pytest.raises(TypeError):
        ops.distill(x, ids.float(), t, loss, st)
    with pytest.raises(TypeError):
        ops.distill(x, ids, t.double(), loss, st)
    with pytest.raises(ValueError):
        ops.distill(x, ids, t[:, :1], loss, st)
    with pytest.raises(ValueError):
        ops.distill(x, ids.expand(4, 2).t().contiguous().t(), t, loss, st)
    with pytest.raises(ValueError):
        ops.distill(x, torch.zeros(4, 257, dtype=torch.int64), torch.zeros(4, 257), loss, st)
    with pytest.raises(ValueError):
        ops.distill(x, ids, t, loss[:3], st)
    with pytest.raises(ValueError):
        ops.distill_shard(x, ids, t, torch.zeros(4, 3), first=0, vocab=32)
    with pytest.raises(ValueError):
        ops.distill_join(torch.zeros(4, 4), ids, t, loss, st, vocab=32)
    with pytest.raises(ValueError):
        ops.distill_backward(x, ids, t, st, x[:, :15])
    with pytest.raises(ValueError):
        ops.distill_backward(x, ids, t, st, x, dloss=loss[:3])
    with pytest.raises(ValueError, match="current device"):
        ops.distill_backward(x, ids, t, st, x)
