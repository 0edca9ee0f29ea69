"""Timed cases of the operators of a training step that stand around its
collectives: layer norm and its gradients, the balance loss over the experts
that a router chose and its gradient, and the loss against a teacher's top
logits over a vocabulary that may be cut into shards, with its gradient.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
with the calls of ``copy_reduce_snac_amd.operators``.  ``exact`` computes it
in binary64, in another way than the plain form does.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
IDS = {"i32": torch.int32, "i64": torch.int64}
ESIZE = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}


def listed():
    return [
        # one new token of a single stream: pure latency, no statistics are kept
        {"name": "norm_token", "op": "norm", "tokens": 1, "width": 8192, "dtype": "bf16", "params": "bf16", "bias": True,
         "stats": False},
        # a training micro-batch or a long prompt
        {"name": "norm_batch", "op": "norm", "tokens": 32768, "width": 4096, "dtype": "bf16", "params": "bf16",
         "bias": True, "stats": True},
        # its gradients: of the rows, and of weight and bias over all tokens
        {"name": "norm_backward", "op": "norm_backward", "tokens": 16384, "width": 4096, "dtype": "bf16",
         "params": "bf16", "bias": True, "grad": "f32"},
        # a small model in binary32 at odd sizes, rows off the lines
        {"name": "norm_backward_ragged", "op": "norm_backward", "tokens": 2049, "width": 1030, "dtype": "f32",
         "params": "f32", "bias": True, "grad": "f32"},
        # the balance of a small, ragged batch over few experts
        {"name": "balance_small", "op": "balance", "tokens": 509, "experts": 60, "topk": 4, "score": "softmax",
         "dtype": "bf16"},
        # the balance of a whole micro-batch over many experts
        {"name": "balance_batch", "op": "balance", "tokens": 32768, "experts": 256, "topk": 8, "score": "sigmoid",
         "dtype": "f32"},
        # its gradient: every logit gets one
        {"name": "balance_backward", "op": "balance_backward", "tokens": 32768, "experts": 128, "topk": 8,
         "score": "softmax", "dtype": "f32"},
        # a few tokens against a teacher's eight best: latency of one long row
        {"name": "distill_few", "op": "distill", "tokens": 7, "vocab": 32768, "shards": 1, "topk": 8,
         "temperature": 1.0, "dtype": "f32", "teacher": "f32", "ids": "i64"},
        # a micro-batch over a large vocabulary, the teacher's 64 best of each token
        {"name": "distill_batch", "op": "distill", "tokens": 4096, "vocab": 131072, "shards": 1, "topk": 64,
         "temperature": 2.0, "dtype": "bf16", "teacher": "bf16", "ids": "i64"},
        # a vocabulary of no round size in four shards of a rank each, and what joins them
        {"name": "distill_shards", "op": "distill", "tokens": 1021, "vocab": 50001, "shards": 4, "topk": 20,
         "temperature": 1.5, "dtype": "f32", "teacher": "f32", "ids": "i64"},
        # the gradient of the micro-batch's logits
        {"name": "distill_backward", "op": "distill_backward", "tokens": 4096, "vocab": 131072, "shards": 1, "topk": 64,
         "temperature": 2.0, "dtype": "bf16", "teacher": "bf16", "ids": "i64"},
        # the gradient of odd rows in binary32
        {"name": "distill_backward_ragged", "op": "distill_backward", "tokens": 509, "vocab": 32003, "shards": 1,
         "topk": 33, "temperature": 1.0, "dtype": "f32", "teacher": "f32", "ids": "i32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "norm_backward", "balance", "balance_backward", "distill", "distill",
                     "distill_backward", "distill_backward"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_backward"):
        width = rng.choice([512, 1024, 2048, 4096, 8192, 16384, rng.randint(64, 6000), rng.randint(64, 6000)])
        tokens = min(_log(rng, 1, 32768), (128 << 20) // (width * ESIZE[dtype]))
        c = {"op": op, "tokens": tokens, "width": width, "dtype": dtype, "params": rng.choice(["f32", "bf16"]),
             "bias": rng.random() < 0.7}
        return {**c, "stats": rng.random() < 0.7} if op == "norm" else {**c, "grad": rng.choice(["f32", "bf16"])}
    if op in ("balance", "balance_backward"):
        experts = _log(rng, 4, 512)
        return {"op": op, "tokens": _log(rng, 1, 32768), "experts": experts, "topk": rng.randint(1, min(10, experts)),
                "score": rng.choice(["softmax", "sigmoid"]), "dtype": dtype}
    shards = rng.choice([1, 1, 1, 2, 4, 8])
    vocab = rng.choice([32768, 65536, 131072, _log(rng, 1000, 160_000), _log(rng, 1000, 160_000)])
    tokens = min(_log(rng, 1, 8192), (512 << 20) // (vocab * ESIZE[dtype]))
    return {"op": op, "tokens": tokens, "vocab": vocab, "shards": shards, "topk": _log(rng, 1, 128),
            "temperature": rng.choice([1.0, 1.5, 2.0, 4.0]), "dtype": dtype, "teacher": rng.choice(["f32", "bf16"]),
            "ids": rng.choice(["i32", "i64"])}


# ------------------------------------------------------------------ inputs

_EPS = 1e-5
_COEFFICIENT = 0.01


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _cuts(c):
    """(first column, columns) of each shard of the vocabulary."""
    per = -(-c["vocab"] // c["shards"])
    return [(r * per, max(0, min(per, c["vocab"] - r * per))) for r in range(c["shards"])]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = c["op"], DTYPES[c["dtype"]]
    s = {"case": c}
    if op in ("norm", "norm_backward"):
        t, w, pt = c["tokens"], c["width"], DTYPES[c["params"]]
        # a residual stream: columns of different sizes and offsets
        size, offset = torch.exp(_normal(g, w) * 0.3), _normal(g, w) * 0.4
        s["x"] = (_normal(g, t, w) * size + offset).to(dt)
        s["weight"] = (1.0 + 0.1 * _normal(g, w)).to(pt)
        s["bias"] = (0.1 * _normal(g, w)).to(pt) if c["bias"] else None
        if op == "norm":
            s["out"] = torch.empty_like(s["x"])
            s["stats"] = torch.empty(t, 2, device="cuda") if c["stats"] else None
        else:
            x = s["x"].double()
            mean = x.mean(dim=1)
            s["stats"] = torch.stack([mean, ((x - mean.unsqueeze(1)).square().mean(dim=1) + _EPS).rsqrt()], dim=1).float()
            s["dout"] = (_normal(g, t, w) * 0.1).to(dt)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = torch.empty(w, dtype=DTYPES[c["grad"]], device="cuda")
            s["dbias"] = torch.empty(w, dtype=DTYPES[c["grad"]], device="cuda") if c["bias"] else None
    elif op in ("balance", "balance_backward"):
        t, e, k = c["tokens"], c["experts"], c["topk"]
        x = _normal(g, t, e) * 1.5 + _normal(g, e) * 0.5
        if t > 16:  # masked experts, and one padding row that is masked as a whole
            x = torch.where(_uniform(g, t, e) < 0.01, torch.full_like(x, -math.inf), x)
            x[t // 3] = -math.inf
        s["logits"] = x.to(dt)
        top = torch.topk(s["logits"].float(), k, dim=1)
        s["chosen"] = torch.where(top.values == -math.inf, torch.full_like(top.indices, -1), top.indices).to(torch.int32)
        s["load"] = torch.empty(2, e, device="cuda")
        if op == "balance":
            s["loss"] = torch.empty(1, device="cuda")
        else:
            s["load"] = _load(c, s["logits"], s["chosen"])
            s["dloss"] = torch.full((1,), 0.75, device="cuda")
            s["dlogits"] = torch.empty_like(s["logits"])
    else:
        t, v, tau = c["tokens"], c["vocab"], c["temperature"]
        live = v - 2  # the last columns pad the vocabulary and are masked
        k = min(c["topk"], live)
        start = (_uniform(g, t, 1) * live).long()
        step = 1 + (_uniform(g, t, 1) * (live // k - 1)).long()
        ids = (start + step * torch.arange(k, device="cuda")) % live
        teacher = torch.sort(8.0 + 3.0 * _normal(g, t, k), dim=1, descending=True).values.to(DTYPES[c["teacher"]])
        z = torch.empty(t, v, dtype=dt, device="cuda").normal_(0.0, 1.5, generator=g)
        z.scatter_(1, ids, (teacher.float() + 0.8 * _normal(g, t, k)).to(dt))
        z[:, live:] = -math.inf
        if t > 16:  # fewer choices for some tokens, and padding tokens without any
            drop = torch.arange(k, device="cuda").unsqueeze(0) >= torch.where(_uniform(g, t, 1) < 0.1, max(1, k // 2), k)
            drop |= _uniform(g, t, 1) < 0.05
            ids = torch.where(drop, torch.full_like(ids, -1), ids)
        s["ids"], s["teacher"] = ids.to(IDS[c["ids"]]), teacher
        s["logits"] = [z] if c["shards"] == 1 else [z[:, a:a + n].contiguous() for a, n in _cuts(c)]
        if op == "distill":
            s["loss"] = torch.empty(t, device="cuda")
            s["stats"] = torch.empty(t, 2, device="cuda")
            s["parts"] = torch.empty(c["shards"], t, 4, device="cuda")
        else:
            top = z.amax(dim=1).float()
            s["stats"] = torch.stack([top, torch.exp((z.float() - top.unsqueeze(1)) / tau).sum(dim=1)], dim=1)
            s["dloss"] = 0.5 + _uniform(g, t)
            s["scale"] = tau * tau / t
            s["dlogits"] = [torch.empty_like(z) for z in s["logits"]]
    return s


# -------------------------------------------------------------------- runs


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
    if op == "norm":
        ops.layer_norm(s["x"], s["weight"], s["bias"], s["out"], eps=_EPS, stats=s["stats"])
        return (s["out"], s["stats"]) if c["stats"] else s["out"]
    if op == "norm_backward":
        ops.layer_norm_backward(s["dout"], s["x"], s["weight"], s["stats"], s["dx"], s["dweight"], s["dbias"], _context())
        return (s["dx"], s["dweight"], s["dbias"]) if c["bias"] else (s["dx"], s["dweight"])
    if op == "balance":
        ops.balance_load(s["logits"], s["chosen"], s["load"], _context(), score=c["score"])
        ops.balance_loss(s["load"], s["loss"], coefficient=_COEFFICIENT)
        return s["load"], s["loss"]
    if op == "balance_backward":
        ops.balance_backward(s["logits"], s["chosen"], s["load"], s["dlogits"], score=c["score"],
                             coefficient=_COEFFICIENT, dloss=s["dloss"])
        return s["dlogits"]
    if op == "distill" and c["shards"] == 1:
        ops.distill(s["logits"][0], s["ids"], s["teacher"], s["loss"], s["stats"], temperature=c["temperature"])
        return s["loss"], s["stats"]
    cuts = _cuts(c)
    if op == "distill":
        for (first, _), z, part in zip(cuts, s["logits"], s["parts"]):
            ops.distill_shard(z, s["ids"], s["teacher"], part, first=first, vocab=c["vocab"], temperature=c["temperature"])
        ops.distill_join(s["parts"], s["ids"], s["teacher"], s["loss"], s["stats"], vocab=c["vocab"],
                         temperature=c["temperature"])
        return s["loss"], s["stats"]
    for (first, _), z, dz in zip(cuts, s["logits"], s["dlogits"]):
        ops.distill_backward(z, s["ids"], s["teacher"], s["stats"], dz, dloss=s["dloss"], scale=s["scale"], first=first,
                             vocab=c["vocab"], temperature=c["temperature"])
    return s["dlogits"]


# ------------------------------------------------------------- plain forms


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt(d.square().mean(dim=1, keepdim=True) + _EPS)
    out = d * rstd * s["weight"].float()
    if s["bias"] is not None:
        out = out + s["bias"].float()
    out = out.to(s["x"].dtype)
    return (out, torch.cat([mean, rstd], dim=1)) if s["case"]["stats"] else out


def _plain_norm_backward(s):
    x, dout = s["x"].float(), s["dout"].float()
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    hat = (x - mean) * rstd
    g = dout * s["weight"].float()
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - hat * (g * hat).mean(dim=1, keepdim=True))
    # sums over all tokens are long ones
    total = [(dout * hat).sum(dim=0, dtype=torch.float64)]
    if s["bias"] is not None:
        total.append(dout.sum(dim=0, dtype=torch.float64))
    return (dx.to(s["x"].dtype), *[v.to(s["dweight"].dtype) for v in total])


def _shares(c, logits):
    """Each token's scores over their sum; zeros where every logit is masked."""
    x = logits.float()
    if c["score"] == "softmax":
        top = x.amax(dim=1, keepdim=True)
        e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    else:
        e = 1.0 / (1.0 + torch.exp(-x))
    total = e.sum(dim=1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e))


def _load(c, logits, chosen):
    """How often each expert was chosen, and the sum of its shares over the tokens with a choice (in binary64:
    a sum over all tokens is a long one)."""
    have = chosen >= 0
    e = c["experts"]
    counts = torch.bincount(torch.where(have, chosen, torch.full_like(chosen, e)).reshape(-1).long(), minlength=e + 1)[:e]
    shares = _shares(c, logits) * have.any(dim=1, keepdim=True)
    return torch.stack([counts.double(), shares.sum(dim=0, dtype=torch.float64)]).float()


def _plain_balance(s):
    c = s["case"]
    load = _load(c, s["logits"], s["chosen"])
    part = load / load.sum(dim=1, keepdim=True).clamp(min=1e-30)
    return load, (_COEFFICIENT * c["experts"] * (part[0] * part[1]).sum()).reshape(1)


def _plain_balance_backward(s):
    c = s["case"]
    p = _shares(c, s["logits"])
    load = s["load"].double()
    total = load.sum(dim=1)
    slope = _COEFFICIENT * c["experts"] * s["dloss"] * (load[0] / (total[0] * total[1]).clamp(min=1e-300))
    # loads that are nearly equal: what is left of them is small
    dot = (p.double() * slope).sum(dim=1, keepdim=True)
    dx = p * (slope - dot).float()
    if c["score"] == "sigmoid":
        dx = dx / (1.0 + torch.exp(s["logits"].float()))
    return torch.where((s["chosen"] >= 0).any(dim=1, keepdim=True), dx, torch.zeros_like(dx)).to(s["logits"].dtype)


def _teacher(s):
    """The teacher's distribution over its choices, the valid ones' columns, and which are valid."""
    have = (s["ids"] >= 0) & (s["ids"] < s["case"]["vocab"])
    t = torch.where(have, s["teacher"].float(), torch.full_like(s["teacher"], -math.inf, dtype=torch.float32))
    top = t.amax(dim=1, keepdim=True)
    e = torch.exp((t - torch.where(top == -math.inf, torch.zeros_like(top), top)) / s["case"]["temperature"])
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-30), torch.where(have, s["ids"], torch.zeros_like(s["ids"])).long()


def _plain_distill(s):
    tau = s["case"]["temperature"]
    z = (s["logits"][0] if len(s["logits"]) == 1 else torch.cat(s["logits"], dim=1)).float()
    top = z.amax(dim=1, keepdim=True)
    total = torch.exp((z - top) / tau).sum(dim=1, keepdim=True)
    q, at = _teacher(s)
    logp = (z.gather(1, at) - top) / tau - torch.log(total)
    loss = torch.where(q > 0, q * (torch.log(q) - logp), torch.zeros_like(q)).sum(dim=1)
    return loss, torch.cat([top, total], dim=1)


def _plain_distill_backward(s):
    c = s["case"]
    tau = c["temperature"]
    q, at = _teacher(s)
    any_choice = q.sum(dim=1, keepdim=True) > 0
    factor = torch.where(any_choice, (s["scale"] / tau * s["dloss"]).unsqueeze(1), torch.zeros_like(q[:, :1]))
    z = (s["logits"][0] if len(s["logits"]) == 1 else torch.cat(s["logits"], dim=1)).float()
    d = torch.exp((z - s["stats"][:, :1]) / tau) / s["stats"][:, 1:]
    d = (d.scatter_add_(1, at, -q) * factor).to(s["logits"][0].dtype)
    return [d] if c["shards"] == 1 else [v.contiguous() for v in d.split([n for _, n in _cuts(c)], dim=1)]


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "balance": _plain_balance,
          "balance_backward": _plain_balance_backward, "distill": _plain_distill,
          "distill_backward": _plain_distill_backward}


# ------------------------------------------------------------ in binary64


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    op = c["op"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + _EPS)
        out = torch.addcmul(torch.zeros_like(x) if s["bias"] is None else s["bias"].double().expand_as(x),
                            (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), s["weight"].double().expand_as(x))
        return (out, torch.stack([mean, rstd], dim=1)) if c["stats"] else out
    if op == "norm_backward":
        mean, rstd = s["stats"].double().unbind(1)
        hat = torch.addcmul(-(mean * rstd).unsqueeze(1), s["x"].double(), rstd.unsqueeze(1))
        dout = s["dout"].double()
        dweight, dbias = torch.linalg.vecdot(dout, hat, dim=0), dout.sum(dim=0)
        dout *= s["weight"].double()
        # the part of the gradient along the row of ones and along hat goes
        dx = dout - dout.mean(dim=1, keepdim=True)
        dx -= hat * (torch.linalg.vecdot(dout, hat, dim=1) / c["width"]).unsqueeze(1)
        dx *= rstd.unsqueeze(1)
        return (dx, dweight, dbias) if c["bias"] else (dx, dweight)
    if op in ("balance", "balance_backward"):
        x = s["logits"].double()
        e = c["experts"]
        # the chosen experts as a matrix of zeros and ones
        hit = torch.zeros_like(x)
        for k in range(c["topk"]):
            at = s["chosen"][:, k].long()
            rows = torch.nonzero(at >= 0).reshape(-1)
            hit[rows, at[rows]] += 1.0
        some = (hit.sum(dim=1, keepdim=True) > 0).double()
        log = x - torch.logsumexp(x, dim=1, keepdim=True) if c["score"] == "softmax" else torch.nn.functional.logsigmoid(x)
        p = torch.exp(log).nan_to_num(0.0)
        if c["score"] == "sigmoid":
            p = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
        p = p * some
        if op == "balance":
            counts, sums = hit.sum(dim=0), p.sum(dim=0)
            loss = _COEFFICIENT * e * torch.dot(counts, sums) / (counts.sum() * sums.sum()).clamp(min=1e-300)
            return torch.stack([counts, sums]), loss.reshape(1)
        counts, sums = s["load"].double()
        up = float(s["dloss"]) * _COEFFICIENT * e * counts / (counts.sum() * sums.sum()).clamp(min=1e-300)
        mean = (p @ up).unsqueeze(1)
        slope = torch.sigmoid(-x) if c["score"] == "sigmoid" else 1.0
        return p * slope * (up - mean)
    return _exact_distill(c, s)


def _exact_distill(c, s):
    tau, t = c["temperature"], c["tokens"]
    have = s["ids"] >= 0
    teacher = torch.where(have, s["teacher"].double() / tau, torch.full_like(s["teacher"], -math.inf, dtype=torch.float64))
    logq = (teacher - torch.logsumexp(teacher, dim=1, keepdim=True)).nan_to_num(-math.inf, neginf=-math.inf)
    q = torch.exp(logq)
    loss, stats = [], []
    dz = [torch.empty(z.shape, dtype=torch.float64, device="cuda") for z in s["logits"]] if c["op"] == "distill_backward" else []
    rows = max(1, (1 << 27) // c["vocab"])
    for a in range(0, t, rows):
        b = min(t, a + rows)
        z = torch.cat([v[a:b] for v in s["logits"]], dim=1).double() / tau
        at = s["ids"][a:b].long().clamp(min=0)
        if c["op"] == "distill":
            lse = torch.logsumexp(z, dim=1, keepdim=True)
            top = z.max(dim=1, keepdim=True).values
            gap = logq[a:b] - (z.gather(1, at) - lse)
            loss.append((q[a:b] * torch.where(q[a:b] > 0, gap, torch.zeros_like(gap))).sum(dim=1))
            stats.append(torch.cat([top * tau, torch.exp(lse - top)], dim=1))
        else:
            p = torch.exp(z - (s["stats"][a:b, :1].double() / tau + torch.log(s["stats"][a:b, 1:].double())))
            target = torch.zeros_like(z).scatter_add_(1, at, q[a:b])
            up = s["dloss"][a:b].double() * s["scale"] / tau * have[a:b].any(dim=1)
            d = (p - target) * up.unsqueeze(1)
            for (first, n), out in zip(_cuts(c), dz):
                out[a:b] = d[:, first:first + n]
    return dz if dz else (torch.cat(loss), torch.cat(stats))


# ----------------------------------------------------------- work of a pass


def work(case):
    c = case
    op, e, t = c["op"], ESIZE[c["dtype"]], c["tokens"]
    if op in ("norm", "norm_backward"):
        w, p = c["width"], ESIZE[c["params"]]
        vectors = 2 if c["bias"] else 1
        if op == "norm":
            return {"bytes": 2 * t * w * e + vectors * w * p + (8 * t if c["stats"] else 0), "flops": 8 * t * w}
        return {"bytes": 3 * t * w * e + w * p + vectors * w * ESIZE[c["grad"]] + 8 * t, "flops": 14 * t * w}
    if op in ("balance", "balance_backward"):
        n, k = c["experts"], c["topk"]
        back = op == "balance_backward"
        return {"bytes": t * n * e * (2 if back else 1) + 4 * t * k + 8 * n + 4, "flops": (10 if back else 6) * t * n}
    v, k = c["vocab"], min(c["topk"], c["vocab"] - 2)
    back = op == "distill_backward"
    choices = t * k * (ESIZE[c["ids"]] + ESIZE[c["teacher"]])
    return {"bytes": t * v * e * (2 if back else 1) + choices + 12 * t, "flops": 5 * t * v}
