"""Timed cases of the operators that stand beside the collectives in a step
of a sharded language model: routing to experts, dispatch and combine around
AllToAllV, the vocabulary-sharded embedding, and the global gradient norm.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
with the calls of ``copy_reduce_snac_amd.operators``.  ``exact`` computes it
in binary64, in another way than the plain form does.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one new token per step of a single stream: pure latency
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 256, "topk": 8, "groups": 8, "topk_groups": 4,
         "score": "sigmoid", "bias": True, "renorm": True, "dtype": "f32"},
        # the router of a whole prompt or training micro-batch, group-limited, with the balance bias
        {"name": "route_prompt", "op": "route", "tokens": 32768, "experts": 256, "topk": 8, "groups": 8,
         "topk_groups": 4, "score": "sigmoid", "bias": True, "renorm": True, "dtype": "f32"},
        # a ragged prefill with few experts, softmax scores kept as they are
        {"name": "route_ragged", "op": "route", "tokens": 4097, "experts": 60, "topk": 4, "groups": 1,
         "topk_groups": 1, "score": "softmax", "bias": False, "renorm": False, "dtype": "bf16"},
        # the router's gradient in training: every logit gets one
        {"name": "route_backward", "op": "route_backward", "tokens": 32768, "experts": 128, "topk": 8, "groups": 1,
         "topk_groups": 1, "score": "softmax", "bias": False, "renorm": False, "dtype": "f32"},
        # a decode batch on its way into AllToAllV
        {"name": "dispatch_decode", "op": "dispatch", "tokens": 32, "experts": 256, "topk": 8, "width": 2048,
         "drop": 0.0, "dtype": "bf16"},
        # a prompt on its way into AllToAllV: each row is sent to eight experts
        {"name": "dispatch_prompt", "op": "dispatch", "tokens": 16384, "experts": 256, "topk": 8, "width": 2048,
         "drop": 0.02, "dtype": "bf16"},
        # what comes back from AllToAllV, odd sizes, rows whose experts were all dropped
        {"name": "combine_ragged", "op": "combine", "tokens": 2049, "experts": 12, "topk": 3, "width": 1030,
         "drop": 0.1, "dtype": "f32"},
        # the gradient of the combine in training: rows for the experts and the router's dweights
        {"name": "combine_backward", "op": "combine_backward", "tokens": 16384, "experts": 64, "topk": 4,
         "width": 2048, "drop": 0.02, "dtype": "bf16"},
        # a decode batch on one vocabulary shard of four: three tokens in four belong to another rank
        {"name": "embedding_decode", "op": "embedding", "tokens": 64, "vocab": 32768, "shards": 4, "width": 8192,
         "dtype": "bf16"},
        # the gradient of the table for a training micro-batch, few tokens making up most of the text
        {"name": "embedding_backward", "op": "embedding_backward", "tokens": 32768, "vocab": 65536, "shards": 1,
         "width": 2048, "dtype": "bf16", "grad": "f32"},
        # the gradients of a small model, or of one layer: many small tensors of both types
        {"name": "clip_small", "op": "clip", "tensors": 96, "elements": 1_000_003},
        # one rank's gradients of a model of some 0.5 G parameters, norms and matrices mixed
        {"name": "clip_large", "op": "clip", "tensors": 300, "elements": 536_870_912},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "dispatch", "combine", "combine_backward", "embedding",
                     "embedding_backward", "embedding_backward", "clip"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _log(rng, 4, 512 // groups)
        keep = rng.randint(max(1, groups // 2), groups)
        return {"op": op, "tokens": _log(rng, 1, 32768), "experts": experts,
                "topk": rng.randint(1, min(10, experts // groups * keep)), "groups": groups, "topk_groups": keep,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "renorm": rng.random() < 0.5, "dtype": dtype}
    if op == "clip":
        return {"op": op, "tensors": _log(rng, 1, 1000), "elements": _log(rng, 5_000, 200_000_000)}
    width = rng.choice([512, 1024, 2048, 4096, 8192, rng.randint(64, 4096), rng.randint(64, 4096)])
    if op in ("embedding", "embedding_backward"):
        vocab = _log(rng, 512, 131072)
        while vocab * width > 134_217_728:
            vocab //= 2
        tokens = min(_log(rng, 1, 65536), 67_108_864 // width)
        c = {"op": op, "tokens": tokens, "vocab": vocab, "shards": rng.choice([1, 1, 2, 8]), "width": width,
             "dtype": dtype}
        return {**c, "grad": rng.choice(["f32", "bf16"])} if op == "embedding_backward" else c
    topk = rng.randint(1, 8)
    experts = _log(rng, max(topk, 4), 512)
    tokens = min(_log(rng, 1, 16384), 134_217_728 // (width * topk))
    return {"op": op, "tokens": max(1, tokens), "experts": experts, "topk": topk, "width": width,
            "drop": rng.choice([0.0, 0.02, 0.3]), "dtype": dtype}


# ------------------------------------------------------------------ inputs


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _slots(c, g):
    """Distinct experts per token, some favoured; a dropped slot is -1, and some tokens lose every slot."""
    t, e, k = c["tokens"], c["experts"], c["topk"]
    ids = (_normal(g, t, e) + _normal(g, e)).topk(k, dim=1).indices.to(torch.int32)
    lost = (_uniform(g, t, k) < c["drop"]) | (_uniform(g, t, 1) < c["drop"] / 4)
    return torch.where(lost, torch.full_like(ids, -1), ids)


def _sort_slots(ids, experts):
    """counts per expert, the row of each slot (-1: dropped) and the slot of each row (-1: unused)."""
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    rows = torch.arange(flat.numel(), device=ids.device)
    kept = key[order] < experts
    row_of_slot = torch.full_like(flat, -1)
    row_of_slot[order] = torch.where(kept, rows, torch.full_like(rows, -1))
    slot_of_row = torch.where(kept, order, torch.full_like(order, -1))
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    return counts.to(torch.int32), row_of_slot.to(torch.int32), slot_of_row.to(torch.int32)


def _tokens(c, g):
    """Token ids over all shards, by a power law over a shuffled vocabulary; this rank holds the second shard
    (the only one where there is one)."""
    n = c["vocab"] * c["shards"]
    rank = (torch.exp(_uniform(g, c["tokens"]).double() * math.log(n + 1.0)) - 1.0).long().clamp(0, n - 1)
    return (rank * 2654435761 + 12345) % n, (c["vocab"] if c["shards"] > 1 else 0)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = c["op"]
    s = {"case": c}
    if op in ("route", "route_backward"):
        t, e, k = c["tokens"], c["experts"], c["topk"]
        x = _normal(g, t, e) * 1.5 + _normal(g, e) * 0.5
        if t > 16:  # masked experts, and one padding row that is masked as a whole
            x = torch.where(_uniform(g, t, e) < 0.01, torch.full_like(x, -math.inf), x)
            x[t // 3] = -math.inf
        s["logits"] = x.to(DTYPES[c["dtype"]])
        s["bias"] = _normal(g, e) * 0.05 if c["bias"] else None
        s["weights"] = torch.empty(t, k, device="cuda")
        s["ids"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
        if op == "route_backward":
            s["ids"] = _choose(c, s["logits"], s["bias"])[1]
            s["dweights"] = _normal(g, t, k)
            s["dlogits"] = torch.empty_like(s["logits"])
    elif op in ("dispatch", "combine", "combine_backward"):
        t, k, w, dt = c["tokens"], c["topk"], c["width"], DTYPES[c["dtype"]]
        s["slots"] = _slots(c, g)
        m = t * k
        if op == "dispatch":
            s["x"] = _normal(g, t, w).to(dt)
            s["counts"] = torch.empty(c["experts"], dtype=torch.int32, device="cuda")
            s["row_of_slot"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
            s["slot_of_row"] = torch.empty(m, dtype=torch.int32, device="cuda")
            s["out"] = torch.zeros(m, w, dtype=dt, device="cuda")
        else:
            s["row_of_slot"] = _sort_slots(s["slots"], c["experts"])[1].view(t, k)
            s["y"] = torch.empty(m, w, dtype=dt, device="cuda").normal_(generator=g)
            s["weights"] = torch.softmax(_normal(g, t, k), dim=1)
            s["out"] = torch.empty(t, w, dtype=dt, device="cuda")
            if op == "combine_backward":
                s["dout"] = _normal(g, t, w).to(dt)
                s["dy"] = torch.zeros(m, w, dtype=dt, device="cuda")
                s["dweights"] = torch.empty(t, k, device="cuda")
    elif op in ("embedding", "embedding_backward"):
        t, v, w, dt = c["tokens"], c["vocab"], c["width"], DTYPES[c["dtype"]]
        s["ids"], s["first"] = _tokens(c, g)
        s["scale"] = math.sqrt(w)
        if op == "embedding":
            s["table"] = torch.empty(v, w, dtype=dt, device="cuda").normal_(0.0, 0.02, generator=g)
            s["out"] = torch.empty(t, w, dtype=dt, device="cuda")
        else:
            s["dout"] = _normal(g, t, w).to(dt)
            s["dtable"] = torch.empty(v, w, dtype=DTYPES[c["grad"]], device="cuda")
    else:
        # two flat buckets; the tensors lie in them one after another, at whatever element they come to
        n = c["elements"]
        half = n // 2
        s["flat"] = [torch.empty(half, dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.01, generator=g),
                     torch.empty(n - half, device="cuda").normal_(0.0, 0.01, generator=g)]
        s["out"] = [torch.empty_like(f) for f in s["flat"]]
        cuts = [_cuts(half, (c["tensors"] + 1) // 2, seed), _cuts(n - half, max(1, c["tensors"] // 2), seed + 1)]
        pairs = [(f[a:b], o[a:b]) for f, o, cut in zip(s["flat"], s["out"], cuts) for a, b in cut]
        s["grads"], s["outs"] = [p[0] for p in pairs], [p[1] for p in pairs]
        s["norm"] = torch.empty(1, device="cuda")
        s["max_norm"] = 1.0
        if own:  # the list of a program's gradients is made once, when its buckets are
            from copy_reduce_snac_amd import operators as ops

            s["list"] = ops.GradList(s["grads"], s["outs"])
    return s


def _cuts(n, k, seed):
    """k pieces of [0, n), of very different lengths: small norms and biases between large matrices."""
    k = min(k, n)
    r = torch.Generator()
    r.manual_seed(seed)
    size = torch.exp(torch.rand(k, generator=r) * 9.0).double()
    ends = (torch.cumsum(size, 0) / size.sum() * (n - k)).long() + torch.arange(1, k + 1)
    ends[-1] = n
    ends = ends.tolist()
    return list(zip([0] + ends[:-1], ends))


# -------------------------------------------------------------------- runs

_SCALE = 2.5


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


_handle = []


def _context():
    """The program's one context, for the operators that need scratch."""
    import copy_reduce_snac_amd as snac

    if not _handle:
        _handle.append(snac.snac_init(1))
    return _handle[0]


def _run_own(s):
    from copy_reduce_snac_amd import operators as ops

    c = s["case"]
    op = c["op"]
    if op == "route":
        ops.route(s["logits"], s["weights"], s["ids"], bias=s["bias"], score=c["score"], groups=c["groups"],
                  topk_groups=c["topk_groups"], renorm=c["renorm"], scale=_SCALE)
        return s["weights"], s["ids"]
    if op == "route_backward":
        ops.route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=c["score"], renorm=c["renorm"],
                           scale=_SCALE)
        return s["dlogits"]
    if op == "dispatch":
        ops.dispatch_plan(s["slots"], s["counts"], s["row_of_slot"], s["slot_of_row"], _context())
        ops.dispatch(s["x"], s["row_of_slot"], s["out"])
        return s["counts"], s["row_of_slot"], s["slot_of_row"], s["out"]
    if op == "combine":
        ops.combine(s["y"], s["row_of_slot"], s["weights"], s["out"])
        return s["out"]
    if op == "combine_backward":
        ops.combine_backward(s["dout"], s["y"], s["row_of_slot"], s["weights"], s["dy"], s["dweights"])
        return s["dy"], s["dweights"]
    if op == "embedding":
        ops.embedding(s["table"], s["ids"], s["out"], first=s["first"], scale=s["scale"])
        return s["out"]
    if op == "embedding_backward":
        ops.embedding_backward(s["dout"], s["ids"], s["dtable"], _context(), first=s["first"], scale=s["scale"])
        return s["dtable"]
    ops.clip_grad_norm(s["list"], s["max_norm"], s["norm"])
    return s["norm"], s["out"]


# ------------------------------------------------------------- plain forms


def _choose(c, logits, bias):
    """The keys in binary64, so that what lies next to a border falls on its right side; the chosen experts."""
    x = logits.double()
    empty = (x == -math.inf).all(dim=1, keepdim=True)
    if c["score"] == "softmax":
        e = torch.exp(x - torch.where(empty, torch.zeros_like(x[:, :1]), x.amax(dim=1, keepdim=True)))
        scores = torch.where(empty, torch.zeros_like(e), e / e.sum(dim=1, keepdim=True))
    else:
        scores = 1.0 / (1.0 + torch.exp(-x))
    key = scores if bias is None else scores + bias.double()
    key = torch.where(x == -math.inf, x, key)
    t, n = x.shape
    g = c["groups"]
    if g > 1:
        best = torch.topk(key.view(t, g, n // g), min(2, n // g), dim=2).values.sum(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : c["topk_groups"]]
        kept = torch.zeros(t, g, dtype=torch.bool, device=x.device)
        kept.scatter_(1, order, (best.gather(1, order) > -math.inf))
        key = torch.where(kept.repeat_interleave(n // g, dim=1), key, torch.full_like(key, -math.inf))
    top = torch.sort(key, dim=1, descending=True, stable=True)
    ids = top.indices[:, : c["topk"]]
    ids = torch.where(top.values[:, : c["topk"]] == -math.inf, torch.full_like(ids, -1), ids)
    return scores, ids.to(torch.int32)


def _plain_route(s):
    c = s["case"]
    scores, ids = _choose(c, s["logits"], s["bias"])
    chosen = scores.float().gather(1, ids.clamp(min=0).long())
    chosen = torch.where(ids < 0, torch.zeros_like(chosen), chosen)
    if c["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        chosen = torch.where(total > 0, chosen / total, torch.zeros_like(chosen))
    return chosen * _SCALE, ids


def _plain_route_backward(s):
    c = s["case"]
    x = s["logits"].float()
    ids = s["ids"]
    at, have = ids.clamp(min=0).long(), ids >= 0
    dw = torch.where(have, s["dweights"] * _SCALE, torch.zeros_like(s["dweights"]))
    zero = torch.zeros_like(x)
    if c["score"] == "softmax":
        chosen = torch.where(have, x.gather(1, at), torch.full_like(dw, -math.inf))
        pool = chosen if c["renorm"] else x
        top = pool.amax(dim=1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        total = torch.exp(pool - top).sum(dim=1, keepdim=True).clamp(min=1e-30)
        r = torch.exp(chosen - top) / total
        dot = (r * dw).sum(dim=1, keepdim=True)
        if c["renorm"]:
            dx = zero.scatter_add(1, at, torch.where(have, r * (dw - dot), torch.zeros_like(dw)))
        else:
            p = torch.exp(x - top) / total
            dx = zero.scatter_add(1, at, r * dw) - p * dot
    else:
        sig = torch.where(have, 1.0 / (1.0 + torch.exp(-x.gather(1, at))), torch.zeros_like(dw))
        far = torch.where(have, 1.0 / (1.0 + torch.exp(x.gather(1, at))), torch.zeros_like(dw))
        if c["renorm"]:
            r = sig / sig.sum(dim=1, keepdim=True).clamp(min=1e-30)
            dx = zero.scatter_add(1, at, r * far * (dw - (r * dw).sum(dim=1, keepdim=True)))
        else:
            dx = zero.scatter_add(1, at, dw * sig * far)
    return dx.to(s["logits"].dtype)


def _plain_dispatch(s):
    c = s["case"]
    counts, row_of_slot, slot_of_row = _sort_slots(s["slots"], c["experts"])
    token = slot_of_row.clamp(min=0).long() // c["topk"]
    out = torch.where((slot_of_row >= 0).unsqueeze(1), s["x"][token], torch.zeros_like(s["x"][:1]))
    return counts, row_of_slot.view(c["tokens"], c["topk"]), slot_of_row, out


def _plain_combine(s):
    rows = s["row_of_slot"]
    w = torch.where(rows >= 0, s["weights"], torch.zeros_like(s["weights"]))
    y = s["y"][rows.clamp(min=0).long()].float()
    return (y * w.unsqueeze(2)).sum(dim=1).to(s["y"].dtype)


def _plain_combine_backward(s):
    rows = s["row_of_slot"]
    t, k = rows.shape
    at = rows.clamp(min=0).long()
    dout = s["dout"].float()
    dw = (s["y"][at].float() * dout.unsqueeze(1)).sum(dim=2)
    token = torch.arange(t * k, device=rows.device) // k
    flat = rows.reshape(-1)
    keep = flat >= 0
    dy = torch.zeros_like(s["y"])
    dy[flat[keep].long()] = (dout[token[keep]] * s["weights"].reshape(-1)[keep].unsqueeze(1)).to(dy.dtype)
    return dy, torch.where(rows >= 0, dw, torch.zeros_like(dw))


def _local(s, v):
    at = s["ids"] - s["first"]
    inside = (at >= 0) & (at < v)
    return torch.where(inside, at, torch.zeros_like(at)), inside


def _plain_embedding(s):
    at, inside = _local(s, s["table"].shape[0])
    rows = s["table"][at].float() * s["scale"]
    return torch.where(inside.unsqueeze(1), rows, torch.zeros_like(rows)).to(s["table"].dtype)


def _plain_embedding_backward(s):
    at, inside = _local(s, s["dtable"].shape[0])
    # a frequent token adds up thousands of rows: long sums go in binary64
    total = torch.zeros(s["dtable"].shape, dtype=torch.float64 if s["dout"].shape[0] > 4096 else torch.float32,
                        device=at.device)
    total.index_add_(0, at[inside], s["dout"][inside].to(total.dtype))
    return (total * s["scale"]).to(s["dtable"].dtype)


def _plain_clip(s):
    total = [f.float().square().sum(dtype=torch.float64) for f in s["flat"]]
    norm = torch.sqrt(torch.stack(total).sum()).float().reshape(1)
    factor = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return norm, [(f.float() * factor).to(f.dtype) for f in s["flat"]]


_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "dispatch": _plain_dispatch,
          "combine": _plain_combine, "combine_backward": _plain_combine_backward, "embedding": _plain_embedding,
          "embedding_backward": _plain_embedding_backward, "clip": _plain_clip}


# ------------------------------------------------------------ in binary64


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    op = c["op"]
    if op in ("route", "route_backward"):
        x = s["logits"].double()
        dead = x == -math.inf
        if c["score"] == "softmax":
            p = torch.where(dead.all(1, keepdim=True), torch.zeros_like(x), torch.softmax(x, dim=1).nan_to_num(0.0))
        else:
            p = torch.sigmoid(x)
        if op == "route":
            return _exact_route(c, p, dead, s["bias"])
        pick = torch.zeros_like(x)
        have = (s["ids"] >= 0).double()
        at = s["ids"].clamp(min=0).long()
        pick.scatter_add_(1, at, have)
        up = torch.zeros_like(x).scatter_add_(1, at, have * s["dweights"].double() * _SCALE)
        # the product rule over all experts, with q the chosen scores (over their sum where they are renormalised)
        q = p * pick
        if c["renorm"]:
            q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
        if c["score"] == "softmax":
            rest = q if c["renorm"] else p
            return q * up - rest * (q * up).sum(1, keepdim=True)
        slope = torch.sigmoid(-x) * pick
        if c["renorm"]:
            up = up - (q * up).sum(1, keepdim=True)
        return (q * slope * up).nan_to_num(0.0)
    if op == "dispatch":
        e, k = c["experts"], c["topk"]
        flat = s["slots"].reshape(-1).long()
        hit = flat.unsqueeze(0) == torch.arange(e, device=flat.device).unsqueeze(1) if flat.numel() * e < 2 ** 28 else None
        if hit is None:
            counts = torch.stack([(flat == i).sum() for i in range(e)])
            slot_of_row = torch.cat([torch.nonzero(flat == i).reshape(-1) for i in range(e)])
        else:
            counts = hit.sum(1)
            slot_of_row = torch.nonzero(hit)[:, 1]
        n = slot_of_row.numel()
        rows = torch.full_like(flat, -1)
        rows[slot_of_row] = torch.arange(n, device=flat.device)
        out = torch.zeros(flat.numel(), c["width"], dtype=torch.float64, device=flat.device)
        out[:n] = s["x"].double()[slot_of_row // k]
        tail = torch.full((flat.numel() - n,), -1, dtype=torch.int64, device=flat.device)
        return (counts.to(torch.int32), rows.view(c["tokens"], k).to(torch.int32),
                torch.cat([slot_of_row, tail]).to(torch.int32), out)
    if op == "combine":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for k in range(c["topk"]):
            r = s["row_of_slot"][:, k].long()
            t = torch.nonzero(r >= 0).reshape(-1)
            out[t] += s["y"][r[t]].double() * s["weights"][t, k].double().unsqueeze(1)
        return out
    if op == "combine_backward":
        dy = torch.zeros(s["dy"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["dweights"].shape, dtype=torch.float64, device="cuda")
        for k in range(c["topk"]):
            r = s["row_of_slot"][:, k].long()
            t = torch.nonzero(r >= 0).reshape(-1)
            d = s["dout"][t].double()
            dy[r[t]] = d * s["weights"][t, k].double().unsqueeze(1)
            dw[t, k] = (d * s["y"][r[t]].double()).sum(1)
        return dy, dw
    if op in ("embedding", "embedding_backward"):
        v = c["vocab"]
        mine = torch.nonzero((s["ids"] >= s["first"]) & (s["ids"] < s["first"] + v)).reshape(-1)
        at = s["ids"][mine] - s["first"]
        if op == "embedding":
            out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
            out[mine] = s["table"][at].double() * s["scale"]
            return out
        # runs of equal tokens, added up a step of their length at a time
        at, order = torch.sort(at)
        out = torch.zeros(s["dtable"].shape, dtype=torch.float64, device="cuda")
        if at.numel() == 0:
            return out
        rows, inverse, counts = torch.unique_consecutive(at, return_inverse=True, return_counts=True)
        place = torch.arange(at.numel(), device="cuda") - (torch.cumsum(counts, 0) - counts)[inverse]
        few = counts[inverse] <= 64
        for step in range(int(min(64, counts.max()))):
            now = torch.nonzero(few & (place == step)).reshape(-1)
            out[at[now]] += s["dout"][mine[order[now]]].double()
        for row, n, end in [(a, b, e) for a, b, e in zip(rows.tolist(), counts.tolist(),
                                                         torch.cumsum(counts, 0).tolist()) if b > 64]:
            out[row] = s["dout"][mine[order[end - n:end]]].double().sum(0)
        return out * s["scale"]
    squares = sum(((f[a:a + (1 << 26)].double()) ** 2).sum() for f in s["flat"] for a in range(0, f.numel(), 1 << 26))
    norm = squares.sqrt().reshape(1)
    factor = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return norm, [f.double() * factor for f in s["flat"]]


def _exact_route(c, p, dead, bias):
    key = p.clone() if bias is None else p + bias.double()
    key[dead] = -math.inf
    t, n = key.shape
    g = c["groups"]
    if g > 1:
        by = key.view(t, g, n // g).sort(dim=2, descending=True).values
        worth = by[:, :, 0] + by[:, :, 1] if n // g > 1 else by[:, :, 0]
        # a group stays if fewer than topk_groups others come before it
        j = torch.arange(g, device=key.device)
        before = (worth.unsqueeze(1) > worth.unsqueeze(2)) | (
            (worth.unsqueeze(1) == worth.unsqueeze(2)) & (j.view(1, 1, g) < j.view(1, g, 1)))
        stays = (before.sum(2) < c["topk_groups"]) & (worth > -math.inf)
        key = key.masked_fill(~stays.unsqueeze(2).expand(t, g, n // g).reshape(t, n), -math.inf)
    weights = torch.zeros(t, c["topk"], dtype=torch.float64, device=key.device)
    ids = torch.full((t, c["topk"]), -1, dtype=torch.int32, device=key.device)
    spot = torch.arange(n, device=key.device).expand(t, n)
    for k in range(c["topk"]):
        top = key.amax(1, keepdim=True)
        at = torch.where(key == top, spot, torch.full_like(spot, n)).amin(1, keepdim=True)
        alive = top > -math.inf
        ids[:, k:k + 1] = torch.where(alive, at, torch.full_like(at, -1)).to(torch.int32)
        weights[:, k:k + 1] = torch.where(alive, p.gather(1, at.clamp(max=n - 1)), torch.zeros_like(top))
        key.scatter_(1, at.clamp(max=n - 1), -math.inf)
    if c["renorm"]:
        total = weights.sum(1, keepdim=True)
        weights = torch.where(total > 0, weights / total, torch.zeros_like(weights))
    return weights * _SCALE, ids


# ----------------------------------------------------------- work of a pass


def work(case):
    c = case
    op, e = c["op"], ESIZE[c.get("dtype", "f32")]
    if op in ("route", "route_backward"):
        t, n, k = c["tokens"], c["experts"], c["topk"]
        back = op == "route_backward"
        return {"bytes": t * n * e * (2 if back else 1) + t * k * 8, "flops": 8 * t * n}
    if op in ("dispatch", "combine", "combine_backward"):
        t, k, w = c["tokens"], c["topk"], c["width"]
        m = round(t * k * (1 - c["drop"]) * (1 - c["drop"] / 4))
        if op == "dispatch":
            return {"bytes": t * k * 12 + 4 * c["experts"] + (t + m) * w * e, "flops": 0}
        if op == "combine":
            return {"bytes": t * k * 8 + (t + m) * w * e, "flops": 2 * m * w}
        return {"bytes": t * k * 12 + (t + 2 * m) * w * e, "flops": 3 * m * w}
    if op == "embedding":
        t, w = c["tokens"], c["width"]
        mine = max(1, t // c["shards"])
        return {"bytes": t * 8 + (t + min(mine, c["vocab"])) * w * e, "flops": mine * w}
    if op == "embedding_backward":
        t, w, v = c["tokens"], c["width"], c["vocab"]
        mine = max(1, t // c["shards"])
        return {"bytes": t * 8 + mine * w * e + v * w * ESIZE[c["grad"]], "flops": mine * w}
    half = c["elements"] // 2
    return {"bytes": 2 * (half * 2 + (c["elements"] - half) * 4), "flops": 3 * c["elements"]}
