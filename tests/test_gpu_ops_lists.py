"""Lists of gradient tensors on the GPU: what a norm may not lie in, and lists
that are sound although their tensors share memory.  Bounds (u = 2^-24): a norm
is rounded once, 1.01 u; a clipped element is off by 5 u."""
from __future__ import annotations

import pytest

from gpu_helpers import gpu_available

U = 2.0 ** -24
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_norm_in_the_list():
    import torch

    import copy_reduce_snac_amd as snac
    from copy_reduce_snac_amd import operators as ops

    x = torch.full((1000,), 3.0, device="cuda")
    out = torch.full((1000,), 5.0, device="cuda")
    y = torch.full((16,), 4.0, device="cuda")
    apart, within = ops.GradList([x, y], [out, y]), ops.GradList([x[:300], x[301:]])
    for lst, norm in [(apart, x[999:]), (apart, out[:1]), (apart, y[7:8]), (within, x[299:300]), (within, x[301:302])]:
        for call in (lambda: ops.grad_norm(lst, norm), lambda: ops.clip_grad_norm(lst, 1.0, norm)):
            with pytest.raises(snac.SnacError) as e:
                call()
            assert e.value.status == snac.SNAC_E_ARG and "norm overlaps" in str(e.value)
    with pytest.raises(snac.SnacError):
        ops.clip_grads(apart, out[3:4], 1.0)
    torch.cuda.synchronize()
    assert bool((x == 3).all()) and bool((out == 5).all()) and bool((y == 4).all())
    ops.clip_grads(apart, x[:1], 1.5)  # a norm that is only read may be a source
    want = 3 * 1.5 / (3 + 1e-6)
    assert bool(((out.double() - want).abs() <= 5 * U * want).all())
    ops.grad_norm(within, x[300:301])  # between two tensors
    assert abs(float(x[300]) - 999 ** 0.5 * 3) <= 1.01 * U * 999 ** 0.5 * 3


def test_one_source_for_two_outputs():
    import torch

    from copy_reduce_snac_amd import operators as ops

    x = torch.full((5000,), 3.0, device="cuda")
    outs = [torch.empty(5000, device="cuda"), torch.empty(4000, device="cuda")]
    norm = torch.empty(1, device="cuda")
    ops.clip_grad_norm(ops.GradList([x, x[1000:]], outs), 0.0, norm)
    want = (9000 * 9.0) ** 0.5
    assert abs(float(norm) - want) <= 1.01 * U * want
    assert not bool(outs[0].any()) and not bool(outs[1].any())


def test_a_list_ends_during_a_capture():
    """The collector ends a list while a graph is captured: the capture goes on and the graph is right."""
    import gc

    import torch

    from copy_reduce_snac_amd import operators as ops

    x = torch.empty(3000, device="cuda")
    out, norm = torch.empty_like(x), torch.empty(1, device="cuda")
    kept, other = ops.GradList([x], [out]), ops.GradList([torch.ones(50, device="cuda")])
    other.itself = other
    x.fill_(1.0)
    ops.clip_grad_norm(kept, 1.0, norm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.grad_norm(kept, norm)
        del other
        gc.collect()
        ops.clip_grad_norm(kept, 1.0, norm)
    for value in (2.0, 7.0, 0.5, 2.0):
        x.fill_(value)
        out.zero_()
        torch.randn(1000, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        ops.clip_grad_norm(kept, 1.0, norm)
        assert torch.equal(got, out) and bool((out > 0).all())
    ops.GradList([x]).close()  # frees the one that ended
    assert ops._ended == []
    kept.close()
