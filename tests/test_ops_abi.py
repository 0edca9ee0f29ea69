"""The operators' C ABI on the CPU: exports, the binding, and every refusal,
which must come before anything touches a GPU."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import copy_reduce_snac_amd as snac

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "snac_ops.h")
E = snac.SNAC_E_ARG
A, B, C, D, F = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000
FAR = 1 << 45


def declared() -> list[str]:
    txt = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(snac_[a-z_0-9]+)\s*\(", txt)))


def test_exports_and_binding():
    names = declared()
    assert len(names) >= 13
    for n in names:
        assert hasattr(snac.lib(), n), f"{n} declared but not exported"
        assert hasattr(snac, n), f"binding lacks {n}"
    assert ctypes.sizeof(snac.snac_router) == 32


def refused(fn, *args, says: str = "") -> None:
    with pytest.raises(snac.SnacError) as e:
        fn(*args)
    assert e.value.status == E, str(e.value)
    assert says in str(e.value), str(e.value)


def r(**kw):
    return snac.router(**{"experts": 16, "topk": 4, **kw})


def test_route_refusals():
    def f(rt, logits=A, ld=16, bias=None, tokens=8, dtype="f32", weights=C, ids=D):
        return (snac.snac_route, rt, logits, ld, bias, tokens, dtype, weights, ids)

    for rt, says in [(r(experts=0), "experts"), (r(experts=1025), "experts"), (r(topk=0), "topk"), (r(topk=17), "topk"),
                     (r(experts=64, topk=33), "topk"), (r(groups=0), "groups"), (r(groups=3), "groups"),
                     (r(experts=130, groups=65), "groups"), (r(groups=4, topk_groups=0), "topk_groups"),
                     (r(groups=4, topk_groups=5), "topk_groups"), (r(groups=8, topk_groups=1), "topk 4"),
                     (r(group_top=3), "group_top"), (r(score=2), "score"), (r(renorm=2), "renorm")]:
        refused(*f(rt), says=says)
    refused(snac.snac_route, None, A, 16, None, 8, "f32", C, D, says="router")
    refused(*f(r(), dtype="u32"), says="dtype")
    refused(*f(r(), ld=15), says="stride")
    refused(*f(r(), logits=0), says="logits")
    refused(*f(r(), logits=A + 2), says="aligned")
    refused(*f(r(), bias=B + 1), says="aligned")
    refused(*f(r(), weights=0), says="weights")
    refused(*f(r(), ids=0), says="ids")
    refused(*f(r(), ids=C + 16), says="overlaps")
    refused(*f(r(), weights=A + 64), says="overlaps")
    refused(*f(r(), bias=C), says="overlaps")
    refused(*f(r(), tokens=snac.SNAC_MAX_BYTES // 64 + 1, weights=FAR, ids=2 * FAR), says="SNAC_MAX_BYTES")
    refused(*f(r(), tokens=(1 << 64) - 1), says="SNAC_MAX_BYTES")
    refused(*f(r(), ld=1 << 62), says="SNAC_MAX_BYTES")
    snac.snac_route(r(), 0, 16, None, 0, "bf16", 0, 0)  # nothing to do


def test_route_backward_refusals():
    def f(rt=None, ld=16, ids=B, dw=C, dtype="f32", dx=D, ld_d=16):
        return (snac.snac_route_backward, rt or r(), A, ld, ids, dw, 8, dtype, dx, ld_d)

    refused(*f(rt=r(topk=17)), says="topk")
    refused(*f(dtype="byte"), says="dtype")
    refused(*f(ld=8), says="stride")
    refused(*f(ld_d=8), says="stride")
    refused(*f(dx=A), says="overlaps")
    refused(*f(dx=C), says="overlaps")
    refused(*f(ids=0), says="ids")
    refused(*f(dx=D + 1), says="aligned")
    snac.snac_route_backward(r(), 0, 16, 0, 0, 0, "f32", 0, 16)


def test_plan_refusals():
    def f(ids=A, size=4, n=64, experts=8, counts=B, rows=C, slots=D):
        return (snac.snac_dispatch_plan, None, ids, size, n, experts, counts, rows, slots)

    refused(*f(size=2), says="id_bytes")
    refused(*f(experts=0), says="experts")
    refused(*f(experts=1025), says="experts")
    refused(*f(n=snac.SNAC_MAX_IDS + 1), says="SNAC_MAX_IDS")
    refused(*f(ids=0), says="ids")
    refused(*f(ids=A + 4, size=8), says="aligned")
    refused(*f(counts=0), says="counts")
    refused(*f(rows=D + 8), says="overlaps")
    refused(*f(), says="ctx")


def test_dispatch_and_combine_refusals():
    def d(x=A, ld=32, rows_of=B, tokens=8, k=2, w=32, dtype="f32", out=C, ld_out=32, rows=16):
        return (snac.snac_dispatch, x, ld, rows_of, tokens, k, w, dtype, out, ld_out, rows)

    refused(*d(dtype="byte"), says="dtype")
    refused(*d(k=0), says="topk")
    refused(*d(k=33), says="topk")
    refused(*d(ld=31), says="stride")
    refused(*d(ld_out=31), says="stride")
    refused(*d(rows=1 << 31), says="rows")
    refused(*d(w=1 << 31, ld=1 << 31, ld_out=1 << 31), says="width")
    refused(*d(x=0), says="x is NULL")
    refused(*d(out=A + 32 * 4), says="overlaps")
    refused(*d(rows_of=C), says="overlaps")
    refused(*d(x=A + 2), says="aligned")
    refused(*d(x=A, ld=64, out=A + 31 * 4, ld_out=64), says="overlaps")  # columns that touch
    snac.snac_dispatch(0, 32, 0, 0, 2, 32, "f32", C, 32, 16)
    snac.snac_dispatch(A, 0, 0, 4, 2, 0, "f32", C, 0, 16)

    def c(y=A, ld=32, rows=16, rows_of=B, w=D, tokens=8, k=2, width=32, dtype="bf16", out=C, ld_out=32):
        return (snac.snac_combine, y, ld, rows, rows_of, w, tokens, k, width, dtype, out, ld_out)

    refused(*c(k=33), says="topk")
    refused(*c(out=A), says="overlaps")
    refused(*c(out=D), says="overlaps")
    refused(*c(y=0), says="y is NULL")
    refused(*c(w=D + 2), says="aligned")
    refused(*c(rows=1 << 32), says="rows")
    snac.snac_combine(0, 32, 0, 0, None, 0, 2, 32, "f32", 0, 32)

    def b(g=A, y=B, rows=16, rows_of=C, w=D, dy=F, ld_dy=32, dw=0x600000):
        return (snac.snac_combine_backward, g, 32, y, 32, rows, rows_of, w, 8, 2, 32, "f32", dy, ld_dy, dw)

    refused(*b(dy=A), says="overlaps")
    refused(*b(dy=B + 32 * 4), says="overlaps")  # y, but shifted
    refused(*b(dy=B, ld_dy=33), says="overlaps")  # y, but with other rows
    refused(*b(dw=D), says="overlaps")
    refused(*b(w=0), says="weights")
    refused(*b(dw=0), says="dweights")


def test_embedding_refusals():
    def f(table=A, ld=32, vocab=16, ids=B, size=8, tokens=8, w=32, dtype="bf16", out=C, ld_out=32):
        return (snac.snac_embedding, table, ld, vocab, 0, ids, size, tokens, w, 1.0, dtype, out, ld_out)

    refused(*f(dtype="u32"), says="dtype")
    refused(*f(size=1), says="id_bytes")
    refused(*f(ld=31), says="stride")
    refused(*f(table=0), says="table")
    refused(*f(ids=B + 4), says="aligned")
    refused(*f(out=A + 64), says="overlaps")
    snac.snac_embedding(0, 32, 0, 0, 0, 8, 0, 32, 1.0, "f32", 0, 32)

    def b(dout=A, dtype="bf16", ids=B, size=4, tokens=8, vocab=16, w=32, dt=C, ld_t=32, gt="f32", acc=0):
        return (snac.snac_embedding_backward, None, dout, 32, dtype, ids, size, tokens, 0, vocab, -1, w, 1.0, dt, ld_t, gt, acc)

    refused(*b(gt="byte"), says="grad_dtype")
    refused(*b(acc=2), says="accumulate")
    refused(*b(tokens=snac.SNAC_MAX_IDS + 1), says="SNAC_MAX_IDS")
    refused(*b(vocab=1 << 30), says="vocab")
    refused(*b(ld_t=16), says="stride")
    refused(*b(dt=A), says="overlaps")
    refused(*b(dt=C + 2), says="aligned")
    refused(*b(), says="ctx")
    assert snac.snac_embedding_scratch(snac.SNAC_MAX_IDS + 1, 16, 32) == 0
    assert snac.snac_embedding_scratch(0, 16, 32) == 0
    assert snac.snac_embedding_scratch(8, 16, 32) >= 8 * 16


def test_grads_refusals():
    refused(snac.snac_grads_init, [A], None, [4], ["u32"], says="dtypes[0]")
    refused(snac.snac_grads_init, [0], None, [4], ["f32"], says="NULL")
    refused(snac.snac_grads_init, [A + 2], None, [4], ["f32"], says="aligned")
    refused(snac.snac_grads_init, [A], [A + 8], [4], ["f32"], says="overlaps")
    refused(snac.snac_grads_init, [A], [0], [4], ["f32"], says="NULL")
    refused(snac.snac_grads_init, [A], None, [snac.SNAC_MAX_BYTES], ["f32"], says="SNAC_MAX_BYTES")
    refused(snac.snac_grads_init, [A], None, [(1 << 64) - 1], ["bf16"], says="SNAC_MAX_BYTES")
    with pytest.raises(ValueError):
        snac.snac_grads_init([A], None, [4, 4], ["f32"])
    refused(snac.snac_grad_norm, None, A, says="grads")
    refused(snac.snac_clip_grads, None, A, 1.0, says="grads")
    refused(snac.snac_clip_grads, None, A, -1.0, says="max_norm")
    refused(snac.snac_clip_grads, None, A, float("nan"), says="max_norm")
    refused(snac.snac_clip_grad_norm, None, -0.5, A, says="max_norm")
    snac.snac_grads_finalize(None)


def test_tensor_level_refusals_on_the_cpu():
    """The tensor-level calls look at shapes, types and strides before devices."""
    import torch

    from copy_reduce_snac_amd import operators as ops

    x = torch.zeros(4, 16)
    w, ids = torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        ops.route(x.double(), w, ids)
    with pytest.raises(TypeError):
        ops.route(x, w, ids.long())
    with pytest.raises(ValueError):
        ops.route(x, w[:3], ids)
    with pytest.raises(ValueError):
        ops.route(torch.zeros(16, 4).t(), w, ids)
    with pytest.raises(ValueError):
        ops.route(x, w, ids, bias=torch.zeros(15))
    with pytest.raises(ValueError):  # right in all but the device
        ops.route(x, w, ids)
    with pytest.raises(ValueError):
        ops.route(torch.zeros(1, 16).expand(4, 16), w, ids)  # rows over one another
    with pytest.raises(ValueError):
        ops.dispatch(x, ids, torch.zeros(8, 15))
    with pytest.raises(TypeError):
        ops.dispatch(x, ids, torch.zeros(8, 16, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        ops.combine(torch.zeros(8, 16), ids.long(), None, x)
    with pytest.raises(ValueError):
        ops.embedding(x, torch.zeros(3, dtype=torch.int64), torch.zeros(4, 16))
    with pytest.raises(TypeError):
        ops.embedding(x, torch.zeros(4), torch.zeros(4, 16))
    with pytest.raises(ValueError):
        ops.GradList([x], [x, x])
    with pytest.raises(ValueError):
        ops.GradList([x])
