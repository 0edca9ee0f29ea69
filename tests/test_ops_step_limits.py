"""Layer norm's scratch, calls of distillation that name a shard without its
vocabulary, and a vocabulary that the example cannot cut, on the CPU."""
from __future__ import annotations

import os
import sys

import pytest

import copy_reduce_snac_amd as snac

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEFAULT = 64 << 20  # staging bytes per rank of a context that names no size


@pytest.mark.parametrize("dtype,size", [("f32", 4), ("bf16", 2)])
def test_layer_norm_scratch_fits_a_default_context(dtype, size):
    """Half of one whatever the tokens, and the sums themselves; 8 bytes a token more for rows above 32 KiB."""
    for width in (1, 64, 100, 128, 255, 1000, 2048, 4096, 5003, 8192, 12288, 16384, 16385, 20001, 1 << 17, 1 << 20, 3000001):
        for tokens in (1, 2, 64, 8191, 8192, 8193, 16384, 32768, 40001, 65536, 131072, 1 << 20, 1 << 22):
            if tokens * width * size > 250 << 30:
                continue
            got = snac.snac_layer_norm_scratch(tokens, width, dtype)
            if width * size <= 32768:
                assert 0 < got <= (32 << 20) + 16 * width + 512, (tokens, width)
            else:
                assert 0 < got <= (32 << 20) + 8 * width + 256 + 8 * tokens, (tokens, width)
    for tokens, width in ((32768, 16384), (65536, 12288), (131072, 8192), (16384, 16384)):
        assert snac.snac_layer_norm_scratch(tokens, width, dtype) <= DEFAULT, (tokens, width)


def test_a_shard_needs_its_vocabulary():
    """Without it every column above the shard would be no choice, and the teacher's distribution another."""
    import torch

    from copy_reduce_snac_amd import operators as ops

    x, st = torch.zeros(4, 16), torch.zeros(4, 2)
    ids, t = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for first in (16, -16):
        with pytest.raises(ValueError, match="vocab"):
            ops.distill_backward(x, ids, t, st, x, first=first)
    with pytest.raises(ValueError, match="current device"):
        ops.distill_backward(x, ids, t, st, x, first=16, vocab=64)
    with pytest.raises(ValueError, match="current device"):
        ops.distill_backward(x, ids, t, st, x)


def test_example_refuses_a_vocabulary_in_uneven_shards():
    """The example's shards are equal: a column that no rank held would be a choice without logits."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import distill_step
    finally:
        sys.path.pop(0)
    with pytest.raises(ValueError, match="vocab"):
        distill_step.DistillStep(ranks=4, tokens=16, width=64, vocab=513)
