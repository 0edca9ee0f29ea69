"""Plain binary64 definitions of the operators of include/snac_ops.h, in
NumPy, row by row.  Gradients are written from the formulas;
tests/test_ops_reference.py holds them against differences of the forwards."""
from __future__ import annotations

import numpy as np

from oracle.bf16 import bf16_to_f32, f32_to_bf16

NEG = -np.inf


def round_to(x, dtype: str):
    """Binary64 -> the element type (bf16 by way of binary32, as the kernels round) -> binary64."""
    f = np.asarray(x, np.float64).astype(np.float32)
    return (bf16_to_f32(f32_to_bf16(f)) if dtype == "bf16" else f).astype(np.float64)


def half_step(dtype: str) -> float:
    """Half a step of the type, relative."""
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def scores(x, score: str):
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        m = np.max(x)
        if m == NEG:
            return np.zeros_like(x)
        e = np.exp(x - m)
        return e / e.sum()


def route(x, topk, score="softmax", groups=1, topk_groups=1, group_top=2, renorm=True, scale=1.0, bias=None):
    """(weights, ids) of one row of logits."""
    x = np.asarray(x, np.float64)
    n = x.size
    s = scores(x, score)
    key = s + (0.0 if bias is None else np.asarray(bias, np.float64))
    key = np.where(x == NEG, NEG, key)

    def order(v):  # descending, NaN first, lower index first
        return sorted(range(len(v)), key=lambda i: (0 if np.isnan(v[i]) else 1, -v[i] if not np.isnan(v[i]) else 0, i))

    kept = range(groups)
    if groups > 1:
        gs = n // groups
        worth = []
        for g in range(groups):
            k = key[g * gs:(g + 1) * gs]
            best = [k[i] for i in order(k)[:min(group_top, gs)]]
            worth.append(best[0] + best[1] if len(best) == 2 else best[0])
        kept = [g for g in order(worth)[:topk_groups] if worth[g] != NEG]
    ok = np.zeros(n, bool)
    for g in kept:
        ok[g * (n // groups):(g + 1) * (n // groups)] = True
    key = np.where(ok, key, NEG)
    ids = [i if key[i] != NEG else -1 for i in order(key)[:topk]]
    chosen = [i for i in ids if i >= 0]
    w = np.zeros(topk)
    if chosen:
        v = chosen_scores(x, s, chosen, score, renorm)
        w[:len(chosen)] = v * scale
    return w, np.array(ids, np.int32)


def chosen_scores(x, s, chosen, score, renorm):
    if not renorm:
        return s[chosen]
    if score == "softmax":
        return scores(x[chosen], "softmax") if np.all(np.isfinite(s)) else s[chosen]
    # logs of the sigmoids, so that very low logits keep their ratios
    with np.errstate(all="ignore"):
        log = -np.logaddexp(0.0, -x[chosen])
        e = np.exp(log - log.max())
    return e / e.sum()


def weights_of(x, ids, score, renorm, scale):
    """Weights of a fixed choice: what the gradient is of."""
    chosen = [int(i) for i in ids if 0 <= i < len(x)]
    w = np.zeros(len(ids))
    if chosen:
        v = chosen_scores(np.asarray(x, np.float64), scores(x, score), chosen, score, renorm) * scale
        w[[k for k, i in enumerate(ids) if 0 <= i < len(x)]] = v
    return w


def route_backward(x, ids, dw, score, renorm, scale):
    """dlogits of one row."""
    x = np.asarray(x, np.float64)
    dx = np.zeros_like(x)
    have = [(int(i), float(d) * scale) for i, d in zip(ids, dw) if 0 <= i < x.size]
    if not have:
        return dx
    at = np.array([i for i, _ in have])
    a = np.array([d for _, d in have])
    s = scores(x, score)
    r = chosen_scores(x, s, at, score, renorm)
    if score == "softmax":
        if renorm:
            dx[at] = r * (a - np.dot(r, a))
        else:
            up = np.zeros_like(x)
            up[at] = a
            dx = s * (up - np.dot(r, a))
    else:
        far = scores(-x[at], "sigmoid")
        dx[at] = r * far * (a - np.dot(r, a)) if renorm else a * r * far
    return dx


def plan(ids, experts):
    """(counts, row_of_slot, slot_of_row) of a flat list of experts."""
    ids = np.asarray(ids).reshape(-1)
    slot = [i for e in range(experts) for i in np.flatnonzero(ids == e)]
    counts = np.array([(ids == e).sum() for e in range(experts)], np.int32)
    row = np.full(ids.size, -1, np.int32)
    back = np.full(ids.size, -1, np.int32)
    row[slot] = np.arange(len(slot))
    back[:len(slot)] = slot
    return counts, row, back


def combine(y, rows, w):
    """Sum of weighted rows, and the sum of the magnitudes (for the bound)."""
    y = np.asarray(y, np.float64)
    t, k = rows.shape
    out, mag = np.zeros((t, y.shape[1])), np.zeros((t, y.shape[1]))
    for i in range(t):
        for j in range(k):
            if 0 <= rows[i, j] < y.shape[0]:
                v = y[rows[i, j]] * (1.0 if w is None else float(w[i, j]))
                out[i] += v
                mag[i] += np.abs(v)
    return out, mag


def embedding_backward(dout, ids, first, vocab, pad, scale):
    """Sums by row, magnitudes and how many tokens each row got."""
    dout = np.asarray(dout, np.float64)
    out, mag, n = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1])), np.zeros(vocab, np.int64)
    for t, i in enumerate(int(v) for v in ids):
        if first <= i < first + vocab and i != pad:
            out[i - first] += dout[t]
            mag[i - first] += np.abs(dout[t])
            n[i - first] += 1
    return out * scale, mag * abs(scale), n
