"""The binary64 references of layer norm, the balance loss and distillation:
their gradients against central differences of their forwards.  A central
difference with h = 1e-5 is off by h^2 / 6 times a third derivative (all below
1000 here, 2e-8) and by rounding / h (1e-10)."""
from __future__ import annotations

import numpy as np
import pytest

import ops_step_reference as ref

H, BOUND = 1e-5, 2e-8


def differences(f, x):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += H
        down[i] -= H
        d[i] = (f(up) - f(down)) / (2 * H)
    return d


@pytest.mark.parametrize("weighted", [False, True])
def test_layer_norm(weighted):
    g = np.random.default_rng(1)
    x, dout = g.normal(size=(3, 7)) + 0.5, g.normal(size=(3, 7))
    w, b = (1 + 0.2 * g.normal(size=7), g.normal(size=7)) if weighted else (None, None)
    stats = np.concatenate(ref.moments(x, 1e-3), axis=1)
    dx, dw, db = ref.layer_norm_backward(dout, x, w, stats)
    loss = lambda x, w, b: float((dout * ref.layer_norm(x, w, b, 1e-3)).sum())  # noqa: E731
    assert np.abs(differences(lambda v: loss(v, w, b), x) - dx).max() < BOUND
    one, zero = (w, b) if weighted else (np.ones(7), np.zeros(7))
    assert np.abs(differences(lambda v: loss(x, v, zero), one) - dw).max() < BOUND
    assert np.abs(differences(lambda v: loss(x, one, v), zero) - db).max() < BOUND


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance(score):
    g = np.random.default_rng(2)
    x = g.normal(size=(5, 6))
    x[1, 2] = -np.inf
    ids = np.array([[0, 3], [1, 1], [-1, 6], [5, -1], [2, 4]])
    load = ref.balance_load(x, ids, score)
    assert load[0].tolist() == [1, 2, 1, 1, 1, 1] and abs(load[1].sum() - 4) < 1e-12
    got = ref.balance_backward(x, ids, load, score, 0.3, 1.7)
    finite = np.where(np.isinf(x), 0.0, x)

    def loss(v):
        v = np.where(np.isinf(x), x, v)
        return 1.7 * ref.balance_loss(ref.balance_load(v, ids, score), 0.3)

    assert np.abs(differences(loss, finite) - got).max() < BOUND
    assert (got[2] == 0).all() and got[1, 2] == 0


def test_balance_by_hand():
    x = np.zeros((4, 4))
    assert abs(ref.balance_loss(ref.balance_load(x, [[0], [1], [2], [3]], "softmax"), 0.5) - 0.5) < 1e-15
    assert ref.balance_loss(ref.balance_load(x, [[-1]] * 4, "softmax"), 0.5) == 0.0
    # all tokens to the one expert that has all shares: as uneven as can be
    x[:, 1] = 50.0
    assert abs(ref.balance_loss(ref.balance_load(x, [[1]] * 4, "softmax"), 0.5) - 2.0) < 1e-12


def test_distill():
    g = np.random.default_rng(3)
    z, t = g.normal(size=(4, 9)), g.normal(size=(4, 3))
    z[0, 8] = -np.inf
    ids = np.array([[1, 4, 7], [2, 2, 5], [-1, 3, 9], [-1, -1, 12]])
    up, tau = np.array([0.5, 1.5, -1.0, 2.0]), 1.7
    loss, m, s = ref.distill(z, ids, t, tau)
    assert loss[3] == 0 and (loss[:3] > 0).all()
    got = ref.distill_backward(z, ids, t, tau, np.stack([m, s], axis=1), up)
    finite = np.where(np.isinf(z), 0.0, z)
    f = lambda v: float((up * ref.distill(np.where(np.isinf(z), z, v), ids, t, tau)[0]).sum())  # noqa: E731
    assert np.abs(differences(f, finite) - got).max() < BOUND
    assert (got[3] == 0).all() and got[0, 8] == 0
    # a choice that comes twice is one with both their parts
    q, _, _ = ref.choices(ids, t, 9, tau)
    p = np.exp(z[1, 2] / tau) / np.exp(z[1] / tau).sum()
    assert abs(got[1, 2] - up[1] / tau * (p - q[1, 0] - q[1, 1])) < 1e-12


def test_distill_by_hand():
    z = np.log(np.array([[0.5, 0.25, 0.25]]))
    loss, m, s = ref.distill(z, [[0, 1]], np.log([[0.75, 0.25]]), 1.0)
    assert abs(loss[0] - (0.75 * np.log(1.5) + 0.25 * np.log(1.0))) < 1e-15
    assert m[0] == z[0, 0] and abs(s[0] - 2.0) < 1e-15
    assert ref.distill(z, [[0, -1]], [[5.0, 5.0]], 1.0)[0][0] == pytest.approx(-np.log(0.5))
    assert np.isinf(ref.distill([[-np.inf, 0.0]], [[0]], [[1.0]], 1.0)[0][0])
    assert ref.distill([[-np.inf, -np.inf]], [[0]], [[1.0]], 1.0)[0][0] == 0.0
