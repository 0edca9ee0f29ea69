"""Lists of gradient tensors on the CPU: overlapping outputs are refused before
anything touches a GPU, and a list's end frees nothing by itself."""
from __future__ import annotations

import pytest

import copy_reduce_snac_amd as snac

A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000


def status(srcs, dsts, counts, types=None):
    """SNAC_E_ARG and what it says, or another status (without a GPU a sound list ends at its first HIP call)."""
    try:
        h = snac.snac_grads_init(srcs, dsts, counts, types or ["f32"] * len(srcs))
    except snac.SnacError as e:
        return e.status, str(e)
    snac.snac_grads_finalize(h)
    return 0, ""


REFUSED = {
    "twice in place": ([A, B, A], None, [4, 4, 4]),
    "views of one buffer in place": ([A, A + 40, A + 60], None, [10, 10, 10]),
    "one inside another": ([A, A + 16], None, [100, 4]),
    "other types": ([A, A + 6], None, [2, 4], ["f32", "bf16"]),
    "one output for two": ([A, B], [C, C], [4, 4]),
    "outputs over one another": ([A, B], [C + 12, C], [4, 4]),
    "an output over another source": ([A, B], [B + 12, D], [4, 4]),
    "an output over another tensor's place": ([A, B], [A, A], [4, 4]),
    "in place, and another tensor's source": ([A, A], [A, B], [4, 4]),
    "the last of many": ([A + 64 * i for i in range(300)] + [A + 64 * 150 + 60], None, [16] * 301),
}


@pytest.mark.parametrize("which", REFUSED)
def test_refused(which):
    st, says = status(*REFUSED[which])
    assert st == snac.SNAC_E_ARG and "overlaps" in says, (st, says)


TAKEN = {
    "neighbours": ([A, A + 16, A + 32], None, [4, 4, 4]),
    "out of order": ([A + 32, A, A + 16], None, [4, 4, 4]),
    "one source for two outputs": ([A, A], [B, C], [4, 4]),
    "sources over one another": ([A, A + 8], [B, C], [4, 4]),
    "some in place": ([A, B], [A, C], [4, 4]),
    "nothing twice": ([A, A, A], None, [0, 4, 0]),
}


@pytest.mark.parametrize("which", TAKEN)
def test_not_refused(which):
    """With nothing but addresses the list is uploaded to a GPU if there is one, and never used."""
    st, says = status(*TAKEN[which])
    assert st != snac.SNAC_E_ARG, says


def test_the_end_of_a_list_touches_no_device(monkeypatch):
    """The collector may end a list while a graph is captured: it is freed when another is made or closed."""
    import gc

    import torch

    from copy_reduce_snac_amd import operators as ops

    made, freed = iter(range(1, 9)), []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(ops, "_raw_stream", lambda device: 77)
    monkeypatch.setattr(ops, "snac_grads_init", lambda *a: next(made))
    monkeypatch.setattr(ops, "snac_grads_finalize", lambda h, stream: freed.append((h, stream)))
    one, two = ops.GradList([]), ops.GradList([])
    one.itself = one  # only the collector finds it
    del one
    gc.collect()
    del two
    assert freed == []
    three, four = ops.GradList([]), ops.GradList([])
    assert sorted(freed) == [(1, 77), (2, 77)]
    del three
    assert len(freed) == 2
    four.close(stream=5)
    assert sorted(freed[2:]) == [(3, 5), (4, 5)]
    four.close()
    del four
    with pytest.raises(ValueError):
        ops.GradList([torch.zeros(4).t() for _ in range(1)], [])  # not made at all
    gc.collect()
    assert len(freed) == 4


def test_lists_left_at_the_end_of_the_program():
    """Lists that live until the interpreter ends, when the module's names are gone already, end without a word."""
    import os
    import subprocess
    import sys

    program = """
import torch
from copy_reduce_snac_amd import operators as ops
torch.cuda.current_device = lambda: 0
ops._raw_stream = lambda device: 0
ops.snac_grads_init = lambda *a: 1
one, two = ops.GradList([]), ops.GradList([])
one.other, two.other = two, one
import sys
sys.modules["torch"].kept = ops.GradList([])
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and p.stderr == "", p.stderr
