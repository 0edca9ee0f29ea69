"""The binary64 references of the operators' tests: their gradients against
central differences of their forwards, and the choice of experts by hand."""
from __future__ import annotations

import numpy as np
import pytest

import ops_reference as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    g = np.random.default_rng(5)
    x = g.normal(size=11) * 1.5
    ids = np.array([7, 2, -1, 9])
    dw = g.normal(size=4)
    got = ref.route_backward(x, ids, dw, score, renorm, 2.5)
    h = 1e-5
    for j in range(x.size):
        up, down = x.copy(), x.copy()
        up[j] += h
        down[j] -= h
        d = np.dot(dw, ref.weights_of(up, ids, score, renorm, 2.5) - ref.weights_of(down, ids, score, renorm, 2.5)) / (2 * h)
        # a central difference is off by h^2 / 6 times a third derivative (all below 100 here) and by rounding / h
        assert abs(d - got[j]) < 1e-8, j


def test_choice_by_hand():
    w, ids = ref.route([0.0, 1.0, 1.0, -np.inf], 3, renorm=False)
    assert ids.tolist() == [1, 2, 0]
    assert np.allclose(w, np.array([np.e, np.e, 1.0]) / (2 * np.e + 1))
    # the bias moves the choice and not the weight
    w, ids = ref.route([0.0, 1.0], 1, score="sigmoid", bias=[1.0, 0.0], renorm=False)
    assert ids.tolist() == [0] and np.allclose(w, 0.5)
    # two groups: the second has the larger sum of two, the first the largest key
    x = [3.0, -9.0, 2.0, 2.0]
    assert ref.route(x, 1, "sigmoid", 2, 1, 2)[1].tolist() == [2]
    assert ref.route(x, 1, "sigmoid", 2, 1, 1)[1].tolist() == [0]
    # nothing left
    w, ids = ref.route([-np.inf] * 4, 2)
    assert ids.tolist() == [-1, -1] and w.tolist() == [0.0, 0.0]


def test_plan_by_hand():
    counts, row, back = ref.plan([2, 0, -1, 2, 5], 3)
    assert counts.tolist() == [1, 0, 2]
    assert row.tolist() == [1, 0, -1, 2, -1]
    assert back.tolist() == [1, 0, 3, -1, -1]
