"""Plain binary64 definitions of layer norm, the balance loss and distillation
(include/snac_ops.h), in NumPy.  Gradients are written from the formulas;
tests/test_ops_step_reference.py holds them against differences of the
forwards."""
from __future__ import annotations

import numpy as np

NEG = -np.inf


def f64(x):
    return np.asarray(x, np.float64)


# ----------------------------------------------------------- layer norm


def moments(x, eps):
    x = f64(x)
    mean = x.mean(axis=1, keepdims=True)
    return mean, 1.0 / np.sqrt(((x - mean) ** 2).mean(axis=1, keepdims=True) + eps)


def layer_norm(x, weight, bias, eps):
    mean, rstd = moments(x, eps)
    out = (f64(x) - mean) * rstd
    if weight is not None:
        out = out * f64(weight)
    return out if bias is None else out + f64(bias)


def layer_norm_backward(dout, x, weight, stats):
    """dx, dweight, dbias."""
    dout, stats = f64(dout), f64(stats)
    h = (f64(x) - stats[:, :1]) * stats[:, 1:]
    g = dout if weight is None else dout * f64(weight)
    dx = stats[:, 1:] * (g - g.mean(axis=1, keepdims=True) - h * (g * h).mean(axis=1, keepdims=True))
    return dx, (dout * h).sum(axis=0), dout.sum(axis=0)


# --------------------------------------------------------- balance loss


def used(ids, experts):
    ids = np.asarray(ids)
    return (ids >= 0) & (ids < experts)


def shares(x, score):
    """Each row's shares; 0 where all is masked."""
    x = f64(x)
    with np.errstate(all="ignore"):
        log = x if score == "softmax" else -np.logaddexp(0.0, -x)
        top = log.max(axis=1, keepdims=True)
        e = np.exp(log - np.where(top == NEG, 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return np.where(total == 0.0, 0.0, e / total)


def balance_load(x, ids, score):
    experts = np.asarray(x).shape[1]
    have = used(ids, experts)
    counts = np.bincount(np.asarray(ids)[have], minlength=experts).astype(np.float64)
    return np.stack([counts, (shares(x, score) * have.any(axis=1, keepdims=True)).sum(axis=0)])


def balance_loss(load, coefficient):
    c, s = f64(load)
    if c.sum() == 0 or s.sum() == 0:
        return 0.0
    return coefficient * c.size * float(np.dot(c / c.sum(), s / s.sum()))


def balance_slope(load, coefficient, dloss):
    c, s = f64(load)
    if c.sum() == 0 or s.sum() == 0:
        return np.zeros_like(c)
    return dloss * coefficient * c.size * c / (c.sum() * s.sum())


def balance_backward(x, ids, load, score, coefficient, dloss):
    a = balance_slope(load, coefficient, dloss)
    p = shares(x, score)
    d = p * (a - (p * a).sum(axis=1, keepdims=True))
    if score == "sigmoid":
        with np.errstate(all="ignore"):
            d = d / (1.0 + np.exp(f64(x)))
    return d * used(ids, a.size).any(axis=1, keepdims=True)


# --------------------------------------------------------- distillation


def choices(ids, t, vocab, tau):
    """q, log q and which choices are valid, by token."""
    ids, t = np.asarray(ids), f64(t)
    ok = (ids >= 0) & (ids < vocab) & (t != NEG)
    with np.errstate(all="ignore"):
        s = np.where(ok, t / tau, NEG)
        top = s.max(axis=1, keepdims=True)
        s = s - np.where(top == NEG, 0.0, top)
        total = np.exp(s).sum(axis=1, keepdims=True)
        logq = s - np.log(np.where(total == 0.0, 1.0, total))
        return np.exp(logq), logq, ok


def distill(z, ids, t, tau):
    """loss, m and S by token."""
    z = f64(z)
    q, logq, ok = choices(ids, t, z.shape[1], tau)
    with np.errstate(all="ignore"):
        m = z.max(axis=1)
        s = np.exp((z - np.where(m == NEG, 0.0, m)[:, None]) / tau).sum(axis=1)
        logp = (z - m[:, None]) / tau - np.log(s)[:, None]
        at = np.where(ok, ids, 0)
        term = np.where(q > 0, q * (logq - np.take_along_axis(logp, at, axis=1)), 0.0)
        loss = term.sum(axis=1)
    part = ok.any(axis=1) & (s != 0.0)
    return np.where(part, loss, 0.0), m, s


def distill_backward(z, ids, t, tau, stats, up):
    """The gradient of the whole vocabulary for upstream factors `up` by token."""
    z, stats = f64(z), f64(stats)
    q, _, ok = choices(ids, t, z.shape[1], tau)
    with np.errstate(all="ignore"):
        p = np.exp((z - stats[:, :1]) / tau) / stats[:, 1:]
    d = p.copy()
    for r in range(z.shape[0]):
        np.subtract.at(d[r], np.asarray(ids)[r][ok[r]], q[r][ok[r]])
    part = ok.any(axis=1) & (stats[:, 1] != 0.0)
    return np.where(part[:, None], d * (f64(up) / tau)[:, None], 0.0)
