"""Tensor-level calls of the operators beside the collectives
(include/snac_ops.h): routing, dispatch and combine around ``all_to_all_v``,
the vocabulary-sharded embedding, the global gradient norm, layer norm, the
experts' balance loss and the loss against a teacher's top logits.

As in ``tensors``: the caller creates the outputs, this module checks shapes,
dtypes and devices and hands pointers and sizes to the library, whose kernels
do all the work; ``stream`` defaults to torch's current stream.  Tensors made
on another stream are the caller's to keep alive and in order.  Matrices may
have any row stride, their last dimension is contiguous.
"""
from __future__ import annotations

import torch

from . import (SNAC_MAX_TEACHER, router, snac_balance_backward, snac_balance_load, snac_balance_loss, snac_clip_grad_norm,
               snac_clip_grads, snac_combine, snac_combine_backward, snac_dispatch, snac_dispatch_plan, snac_distill,
               snac_distill_backward, snac_distill_join, snac_distill_shard, snac_embedding, snac_embedding_backward,
               snac_grad_norm, snac_grads_finalize, snac_grads_init, snac_layer_norm, snac_layer_norm_backward,
               snac_route, snac_route_backward)
from . import teacher as teacher_of

_FLOAT = {torch.bfloat16: "bf16", torch.float32: "f32"}
_ID = {torch.int32: 4, torch.int64: 8}


# torch's current stream of a device as a hipStream_t: torch.cuda.current_stream()
# makes a Stream object for it, which takes longer (2.5 us) than a call's other checks
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device: int):
    if stream is not None:
        return stream
    return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device)


def _float(t, what: str) -> str:
    name = _FLOAT.get(t.dtype)
    if name is None:
        raise TypeError(f"{what} must be bfloat16 or float32, not {t.dtype}")
    return name


def _ids(t, what: str) -> int:
    size = _ID.get(t.dtype)
    if size is None:
        raise TypeError(f"{what} must be int32 or int64, not {t.dtype}")
    return size


def _device(what: str, first, *others) -> int:
    """The tensors' device, which has to be the current one."""
    device = first.get_device()
    if device < 0 or device != torch.cuda.current_device():
        raise ValueError(f"{what}: every tensor must be on the current device, not on {first.device}")
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{what}: every tensor must be on the current device, not on {t.device}")
    return device


def _matrix(t, what: str) -> int:
    """Row stride of a matrix with contiguous rows."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must have two dimensions, not {len(shape)}")
    rows, width = shape
    ld, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    if rows < 2:
        return width
    if ld < width:
        raise ValueError(f"{what}: rows overlap")
    return ld


def _packed(t, shape, dtype, what: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _pair(a, b, what: str) -> None:
    if a.dtype != b.dtype:
        raise TypeError(f"{what} must have the same dtype, not {a.dtype} and {b.dtype}")


def route(logits, weights, ids, *, bias=None, score: str = "softmax", groups: int = 1, topk_groups: int = 1,
          group_top: int = 2, renorm: bool = True, scale: float = 1.0, stream=None) -> None:
    """Choose ``ids.shape[1]`` experts for each row of ``logits`` [tokens,
    experts] into ``ids`` (int32) and ``weights`` (float32), both [tokens,
    topk]; ``bias`` [experts] (float32) moves the choice only.  snac_router in
    the C header says how; a masked logit (-inf) is never chosen."""
    ld = _matrix(logits, "route: logits")
    dt = _float(logits, "route: logits")
    t, e = logits.shape
    if ids.dim() != 2:
        raise ValueError("route: ids must have two dimensions")
    k = ids.shape[1]
    _packed(ids, (t, k), torch.int32, "route: ids")
    _packed(weights, (t, k), torch.float32, "route: weights")
    if bias is not None:
        _packed(bias, (e,), torch.float32, "route: bias")
    on = _device("route", logits, weights, ids, bias)
    snac_route(router(e, k, score, groups, topk_groups, group_top, renorm, scale), logits, ld, bias, t, dt, weights,
               ids, _stream(stream, on))


def route_backward(logits, ids, dweights, dlogits, *, score: str = "softmax", renorm: bool = True, scale: float = 1.0,
                   stream=None) -> None:
    """``dlogits`` [tokens, experts] from the gradient of the weights that
    ``route`` gave for ``ids``."""
    ld, ld_d = _matrix(logits, "route_backward: logits"), _matrix(dlogits, "route_backward: dlogits")
    dt = _float(logits, "route_backward: logits")
    t, e = logits.shape
    if ids.dim() != 2 or dlogits.shape != logits.shape:
        raise ValueError("route_backward: ids must have two dimensions and dlogits the shape of logits")
    _pair(logits, dlogits, "route_backward: logits and dlogits")
    k = ids.shape[1]
    _packed(ids, (t, k), torch.int32, "route_backward: ids")
    _packed(dweights, (t, k), torch.float32, "route_backward: dweights")
    on = _device("route_backward", logits, ids, dweights, dlogits)
    snac_route_backward(router(e, k, score, 1, 1, 1, renorm, scale), logits, ld, ids, dweights, t, dt, dlogits, ld_d,
                        _stream(stream, on))


def dispatch_plan(ids, counts, row_of_slot, slot_of_row, handle, stream=None) -> None:
    """The packed order of the slots of ``ids`` [tokens, topk] (int32 or int64)
    by expert: ``counts`` [experts], ``row_of_slot`` [tokens, topk] (-1:
    dropped), ``slot_of_row`` [tokens * topk] (-1: unused), all int32.
    ``handle`` is a context of ``snac_init``; its staging rings are scratch."""
    size = _ids(ids, "dispatch_plan: ids")
    if not ids.is_contiguous():
        raise ValueError("dispatch_plan: ids must be contiguous")
    n = ids.numel()
    if counts.dim() != 1:
        raise ValueError("dispatch_plan: counts must have one dimension")
    _packed(counts, counts.shape, torch.int32, "dispatch_plan: counts")
    _packed(row_of_slot, ids.shape, torch.int32, "dispatch_plan: row_of_slot")
    _packed(slot_of_row, (n,), torch.int32, "dispatch_plan: slot_of_row")
    on = _device("dispatch_plan", ids, counts, row_of_slot, slot_of_row)
    snac_dispatch_plan(handle, ids, size, n, counts.shape[0], counts, row_of_slot, slot_of_row, _stream(stream, on))


def _slots(row_of_slot, tokens: int, what: str) -> int:
    if row_of_slot.dim() != 2:
        raise ValueError(f"{what}: row_of_slot must have two dimensions")
    k = row_of_slot.shape[1]
    _packed(row_of_slot, (tokens, k), torch.int32, f"{what}: row_of_slot")
    return k


def dispatch(x, row_of_slot, out, stream=None) -> None:
    """out[row_of_slot[t, k]] = x[t]; rows of ``out`` that no slot names stay
    as they are.  Its gradient is ``combine`` without weights."""
    ld_x, ld_out = _matrix(x, "dispatch: x"), _matrix(out, "dispatch: out")
    dt = _float(x, "dispatch: x")
    _pair(x, out, "dispatch: x and out")
    t, w = x.shape
    k = _slots(row_of_slot, t, "dispatch")
    if out.shape[1] != w:
        raise ValueError("dispatch: x and out must have rows of the same width")
    on = _device("dispatch", x, row_of_slot, out)
    snac_dispatch(x, ld_x, row_of_slot, t, k, w, dt, out, ld_out, out.shape[0], _stream(stream, on))


def combine(y, row_of_slot, weights, out, stream=None) -> None:
    """out[t] = sum over k of weights[t, k] * y[row_of_slot[t, k]]; ``weights``
    (float32) may be None for a plain sum."""
    ld_y, ld_out = _matrix(y, "combine: y"), _matrix(out, "combine: out")
    dt = _float(y, "combine: y")
    _pair(y, out, "combine: y and out")
    t, w = out.shape
    k = _slots(row_of_slot, t, "combine")
    if y.shape[1] != w:
        raise ValueError("combine: y and out must have rows of the same width")
    if weights is not None:
        _packed(weights, (t, k), torch.float32, "combine: weights")
    on = _device("combine", y, row_of_slot, weights, out)
    snac_combine(y, ld_y, y.shape[0], row_of_slot, weights, t, k, w, dt, out, ld_out, _stream(stream, on))


def combine_backward(dout, y, row_of_slot, weights, dy, dweights, stream=None) -> None:
    """dy[row_of_slot[t, k]] = weights[t, k] * dout[t] (other rows stay as they
    are; ``dy`` may be ``y``) and dweights[t, k] = <dout[t], y[row]>."""
    ld_g, ld_y, ld_dy = (_matrix(m, "combine_backward: " + n) for m, n in ((dout, "dout"), (y, "y"), (dy, "dy")))
    dt = _float(y, "combine_backward: y")
    _pair(y, dout, "combine_backward: y and dout")
    _pair(y, dy, "combine_backward: y and dy")
    t, w = dout.shape
    k = _slots(row_of_slot, t, "combine_backward")
    if y.shape[1] != w or dy.shape != y.shape:
        raise ValueError("combine_backward: rows of different widths, or dy without the shape of y")
    _packed(weights, (t, k), torch.float32, "combine_backward: weights")
    _packed(dweights, (t, k), torch.float32, "combine_backward: dweights")
    on = _device("combine_backward", dout, y, row_of_slot, weights, dy, dweights)
    snac_combine_backward(dout, ld_g, y, ld_y, y.shape[0], row_of_slot, weights, t, k, w, dt, dy, ld_dy, dweights,
                          _stream(stream, on))


def embedding(table, ids, out, *, first: int = 0, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t] - first], zeros for the ids of other
    shards; ``ids`` (int32 or int64) and ``out`` agree in all but out's last
    dimension, the width."""
    ld = _matrix(table, "embedding: table")
    dt = _float(table, "embedding: table")
    _pair(table, out, "embedding: table and out")
    v, w = table.shape
    n, flat = _tokens(ids, out, w, "embedding", "out")
    size = _ids(ids, "embedding: ids")
    on = _device("embedding", table, ids, out)
    snac_embedding(table, ld, v, first, ids, size, n, w, scale, dt, out, flat, _stream(stream, on))


def _tokens(ids, rows, width: int, what: str, name: str):
    """Number of ids, and the row stride of the tensor with a row for each."""
    if rows.shape != (*ids.shape, width):
        raise ValueError(f"{what}: {name} must have shape {(*ids.shape, width)}, not {tuple(rows.shape)}")
    if not ids.is_contiguous():
        raise ValueError(f"{what}: ids must be contiguous")
    if rows.dim() == 2:
        return ids.numel(), _matrix(rows, f"{what}: {name}")
    if not rows.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous unless it is a matrix")
    return ids.numel(), width


def embedding_backward(dout, ids, dtable, handle, *, first: int = 0, pad: int | None = None, scale: float = 1.0,
                       accumulate: bool = False, stream=None) -> None:
    """The gradient of the shard ``dtable`` [vocab, width] (bfloat16 or
    float32, whatever dout's type): scale times the sum of the rows of
    ``dout`` whose id is the row's; ids equal to ``pad`` have none.  Written
    whole, or with ``accumulate`` added to what is there.  ``handle`` is a
    context of ``snac_init`` whose staging rings hold
    ``snac_embedding_scratch`` bytes."""
    ld_t = _matrix(dtable, "embedding_backward: dtable")
    dt, gt = _float(dout, "embedding_backward: dout"), _float(dtable, "embedding_backward: dtable")
    v, w = dtable.shape
    n, ld = _tokens(ids, dout, w, "embedding_backward", "dout")
    size = _ids(ids, "embedding_backward: ids")
    on = _device("embedding_backward", dout, ids, dtable)
    # an id just below the shard is in no row of it
    pad_id = first - 1 if pad is None else pad
    snac_embedding_backward(handle, dout, ld, dt, ids, size, n, first, v, pad_id, w, scale, dtable, ld_t, gt,
                            int(accumulate), _stream(stream, on))


# Lists that ended without close().  The collector may end one at any time, also
# while a graph is captured, where waiting for a stream or freeing memory would
# end the capture: they are freed at the next call that allows both.
_ended: list[int] = []


def _free_ended(stream) -> None:
    while _ended:
        snac_grads_finalize(_ended.pop(), stream)


class GradList:
    """A fixed list of gradient tensors (bfloat16 and float32, contiguous, any
    shapes) for the norm and clipping; ``outs`` receives the clipped ones, by
    default the tensors themselves.  An output overlaps no other tensor of the
    list (so none is listed twice in place), and ``norm`` none of them.  It
    keeps the tensors alive and reads them where they lie at each call, so it
    is for gradients that stay in place (``zero_grad(set_to_none=False)``, or
    buckets): making one takes 0.15 to 0.6 ms and waits for the stream.
    ``close()`` waits for the stream and frees it.  Making and closing lists is
    not to be captured; a list that ends without ``close()`` is freed when the
    next one is made or closed, so it may end at any time."""

    def __init__(self, grads, outs=None, stream=None):
        self._h = None
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        every = self.grads + (self.outs or [])
        if self.outs is not None and len(self.outs) != len(self.grads):
            raise ValueError(f"GradList: {len(self.grads)} tensors but {len(self.outs)} outputs")
        self.device = _device("GradList", *every) if every else torch.cuda.current_device()
        for t in every:
            if not t.is_contiguous():
                raise ValueError("GradList: tensors must be contiguous")
        types = [_float(t, "GradList: a tensor") for t in self.grads]
        for g, o in zip(self.grads, self.outs or []):
            _pair(g, o, "GradList: a tensor and its output")
            if g.numel() != o.numel():
                raise ValueError("GradList: a tensor and its output differ in length")
        on = _stream(stream, self.device)
        _free_ended(on)
        self._h = snac_grads_init(self.grads, self.outs, [t.numel() for t in self.grads], types, on)

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("GradList: closed")
        return self._h

    def close(self, stream=None) -> None:
        on = _stream(stream, self.device)
        h, self._h = self._h, None
        if h is not None:
            snac_grads_finalize(h, on)
        _free_ended(on)

    def __del__(self, ended=_ended):  # bound here: the module's names go before its last lists do
        h = getattr(self, "_h", None)
        if h is not None:
            ended.append(h)


def _scalar(norm, what: str) -> int:
    if norm.numel() != 1 or norm.dtype != torch.float32:
        raise ValueError(f"{what}: norm must be one float32")
    return _device(what, norm)


def grad_norm(grads: GradList, norm, stream=None) -> None:
    """norm[0] = the 2-norm of all elements of the list."""
    on = _scalar(norm, "grad_norm")
    snac_grad_norm(grads.handle, norm, _stream(stream, on))


def clip_grads(grads: GradList, norm, max_norm: float, stream=None) -> None:
    """The list's outputs = its tensors * min(1, max_norm / (norm + 1e-6))."""
    on = _scalar(norm, "clip_grads")
    snac_clip_grads(grads.handle, norm, max_norm, _stream(stream, on))


def clip_grad_norm(grads: GradList, max_norm: float, norm, stream=None) -> None:
    """``grad_norm`` into ``norm``, then ``clip_grads`` by it."""
    on = _scalar(norm, "clip_grad_norm")
    snac_clip_grad_norm(grads.handle, max_norm, norm, _stream(stream, on))


# the calls below build their messages where they raise: a formatted string takes
# as long as the check that it is for
def _vector(t, shape, what: str, name: str) -> str:
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous with shape {tuple(shape)}, not {tuple(t.shape)}")
    return _FLOAT.get(t.dtype) or _float(t, f"{what}: {name}")


def _vectors(a, b, width: int, what: str, name_a: str, name_b: str) -> str:
    """The common type of two vectors that may be None (float32 where both are)."""
    dt = None if a is None else _vector(a, (width,), what, name_a)
    if b is None:
        return dt or "f32"
    dt_b = _vector(b, (width,), what, name_b)
    if dt is not None and dt != dt_b:
        raise TypeError(f"{what}: {name_a} and {name_b} must have the same dtype, not {a.dtype} and {b.dtype}")
    return dt_b


def layer_norm(x, weight, bias, out, *, eps: float = 1e-5, stats=None, stream=None) -> None:
    """Each row of ``x`` [tokens, width] less its mean, over its deviation,
    times ``weight`` plus ``bias`` ([width], bfloat16 or float32, each may be
    None); ``out`` may be ``x``.  ``stats`` [tokens, 2] (float32) receives mean
    and 1 / deviation for the gradient; a pass without one leaves it out."""
    ld_x, ld_out = _matrix(x, "layer_norm: x"), _matrix(out, "layer_norm: out")
    dt = _float(x, "layer_norm: x")
    _pair(x, out, "layer_norm: x and out")
    t, w = x.shape
    if out.shape != x.shape:
        raise ValueError("layer_norm: out must have the shape of x")
    pt = _vectors(weight, bias, w, "layer_norm", "weight", "bias")
    if stats is not None:
        _packed(stats, (t, 2), torch.float32, "layer_norm: stats")
    on = _device("layer_norm", x, weight, bias, out, stats)
    snac_layer_norm(x, ld_x, weight, bias, pt, t, w, eps, dt, out, ld_out, stats, _stream(stream, on))


def layer_norm_backward(dout, x, weight, stats, dx, dweight, dbias, handle=None, *, accumulate: bool = False,
                        stream=None) -> None:
    """``dx`` (may be ``dout``) and the sums over the tokens ``dweight`` and
    ``dbias`` [width] (bfloat16 or float32, each may be None), written or with
    ``accumulate`` added to.  ``stats`` is ``layer_norm``'s.  ``handle`` is a
    context of ``snac_init`` whose staging rings hold
    ``snac_layer_norm_scratch`` bytes; without dweight and dbias rows of up to
    32 KiB need none."""
    ld_g, ld_x = _matrix(dout, "layer_norm_backward: dout"), _matrix(x, "layer_norm_backward: x")
    ld_dx = _matrix(dx, "layer_norm_backward: dx")
    dt = _float(x, "layer_norm_backward: x")
    _pair(x, dout, "layer_norm_backward: x and dout")
    _pair(x, dx, "layer_norm_backward: x and dx")
    t, w = x.shape
    if dout.shape != x.shape or dx.shape != x.shape:
        raise ValueError("layer_norm_backward: dout and dx must have the shape of x")
    pt = _vectors(weight, None, w, "layer_norm_backward", "weight", "")
    gt = _vectors(dweight, dbias, w, "layer_norm_backward", "dweight", "dbias")
    _packed(stats, (t, 2), torch.float32, "layer_norm_backward: stats")
    on = _device("layer_norm_backward", dout, x, weight, stats, dx, dweight, dbias)
    snac_layer_norm_backward(handle, dout, ld_g, x, ld_x, weight, pt, stats, t, w, dt, dx, ld_dx, dweight, dbias, gt,
                             int(accumulate), _stream(stream, on))


def _chosen(logits, ids, what: str):
    """Row stride, type, tokens, experts and choices of a router's logits and ids."""
    ld = _matrix(logits, what)
    dt = _FLOAT.get(logits.dtype) or _float(logits, f"{what}: logits")
    t, e = logits.shape
    if ids.dim() != 2 or ids.shape[0] != t or not ids.is_contiguous():
        raise ValueError(f"{what}: ids must be contiguous with shape [{t}, choices], not {tuple(ids.shape)}")
    if ids.dtype != torch.int32:
        raise TypeError(f"{what}: ids must be int32, not {ids.dtype}")
    return ld, dt, t, e, ids.shape[1]


def balance_load(logits, ids, load, handle, *, score: str = "softmax", stream=None) -> None:
    """``load`` [2, experts] (float32): how many slots of ``ids`` [tokens, topk]
    (int32, what ``route`` chose; others than 0 .. experts - 1 are not in use)
    each expert got, and the sum of its shares of the tokens' scores.  Padding
    tokens, those without an id in use, have no part.  With tokens on several
    ranks an ``all_reduce`` of their loads gives the common one.  ``handle`` is
    a context of ``snac_init``; its staging rings are scratch."""
    ld, dt, t, e, k = _chosen(logits, ids, "balance_load")
    _packed(load, (2, e), torch.float32, "balance_load: load")
    on = _device("balance_load", logits, ids, load)
    snac_balance_load(handle, router(e, k, score), logits, ld, ids, t, dt, load, _stream(stream, on))


def balance_loss(load, loss, *, coefficient: float = 1.0, stream=None) -> None:
    """loss[0] = coefficient * experts * sum of the experts' parts of the slots
    times their parts of the shares: ``coefficient`` where they are even."""
    if load.dim() != 2:
        raise ValueError("balance_loss: load must have two dimensions")
    e = load.shape[1]
    _packed(load, (2, e), torch.float32, "balance_loss: load")
    if loss.numel() != 1 or loss.dtype != torch.float32:
        raise ValueError("balance_loss: loss must be one float32")
    on = _device("balance_loss", load, loss)
    snac_balance_loss(load, e, coefficient, loss, _stream(stream, on))


def balance_backward(logits, ids, load, dlogits, *, score: str = "softmax", coefficient: float = 1.0, dloss=None,
                     accumulate: bool = False, stream=None) -> None:
    """``dlogits`` [tokens, experts], written or with ``accumulate`` added to
    (what ``route_backward`` left), for the ``load`` that the loss was made of
    and ``dloss`` (one float32 on the device, None: 1)."""
    ld, dt, t, e, k = _chosen(logits, ids, "balance_backward")
    ld_d = _matrix(dlogits, "balance_backward: dlogits")
    _pair(logits, dlogits, "balance_backward: logits and dlogits")
    if dlogits.shape != logits.shape:
        raise ValueError("balance_backward: dlogits must have the shape of logits")
    _packed(load, (2, e), torch.float32, "balance_backward: load")
    if dloss is not None and (dloss.numel() != 1 or dloss.dtype != torch.float32):
        raise ValueError("balance_backward: dloss must be one float32")
    on = _device("balance_backward", logits, ids, load, dloss, dlogits)
    snac_balance_backward(router(e, k, score), logits, ld, ids, load, coefficient, dloss, t, dt, dlogits, ld_d,
                          int(accumulate), _stream(stream, on))


def _teacher(ids, logits, tokens: int, vocab: int, temperature: float, what: str):
    size = _ID.get(ids.dtype) or _ids(ids, f"{what}: ids")
    dt = _FLOAT.get(logits.dtype) or _float(logits, f"{what}: teacher")
    shape = ids.shape
    if len(shape) != 2 or shape[0] != tokens or logits.shape != shape:
        raise ValueError(f"{what}: ids and teacher must have shape [{tokens}, choices], not {tuple(ids.shape)} and "
                         f"{tuple(logits.shape)}")
    if not (ids.is_contiguous() and logits.is_contiguous()):
        raise ValueError(f"{what}: ids and teacher must be contiguous")
    if not 1 <= shape[1] <= SNAC_MAX_TEACHER:
        raise ValueError(f"{what}: {shape[1]} choices outside 1..{SNAC_MAX_TEACHER}")
    return teacher_of(ids, size, logits, dt, shape[1], vocab, temperature)


def distill(logits, ids, teacher, loss, stats, *, temperature: float = 1.0, stream=None) -> None:
    """``loss`` [tokens] = the divergence of softmax(``logits`` / temperature)
    [tokens, vocab] from the softmax of a teacher's top logits ``teacher``
    [tokens, choices] (bfloat16 or float32) for the columns ``ids`` (int32 or
    int64; others than 0 .. vocab - 1 are no choices, a token without any has
    loss 0).  ``stats`` [tokens, 2] is for the gradient; both float32.
    snac_teacher in the C header has the formulas."""
    ld = _matrix(logits, "distill: logits")
    dt = _float(logits, "distill: logits")
    t, v = logits.shape
    h = _teacher(ids, teacher, t, v, temperature, "distill")
    _packed(loss, (t,), torch.float32, "distill: loss")
    _packed(stats, (t, 2), torch.float32, "distill: stats")
    on = _device("distill", logits, ids, teacher, loss, stats)
    snac_distill(h, logits, ld, t, dt, loss, stats, _stream(stream, on))


def distill_shard(logits, ids, teacher, part, *, first: int, vocab: int, temperature: float = 1.0, stream=None) -> None:
    """``part`` [tokens, 4] (float32) of a rank that holds columns ``first`` to
    first + logits.shape[1] - 1 of a vocabulary of ``vocab`` columns; the ranks'
    parts, brought together by an ``all_gather``, go to ``distill_join``."""
    ld = _matrix(logits, "distill_shard: logits")
    dt = _float(logits, "distill_shard: logits")
    t, w = logits.shape
    h = _teacher(ids, teacher, t, vocab, temperature, "distill_shard")
    _packed(part, (t, 4), torch.float32, "distill_shard: part")
    on = _device("distill_shard", logits, ids, teacher, part)
    snac_distill_shard(h, logits, ld, first, w, t, dt, part, _stream(stream, on))


def distill_join(parts, ids, teacher, loss, stats, *, vocab: int, temperature: float = 1.0, stream=None) -> None:
    """``loss`` [tokens] and ``stats`` [tokens, 2] of the shards' ``parts``
    [shards, tokens, 4]."""
    if parts.dim() != 3:
        raise ValueError("distill_join: parts must have three dimensions")
    n, t = parts.shape[:2]
    _packed(parts, (n, t, 4), torch.float32, "distill_join: parts")
    h = _teacher(ids, teacher, t, vocab, temperature, "distill_join")
    _packed(loss, (t,), torch.float32, "distill_join: loss")
    _packed(stats, (t, 2), torch.float32, "distill_join: stats")
    on = _device("distill_join", parts, ids, teacher, loss, stats)
    snac_distill_join(h, parts, n, t, loss, stats, _stream(stream, on))


def distill_backward(logits, ids, teacher, stats, dlogits, *, dloss=None, scale: float = 1.0, first: int = 0,
                     vocab: int | None = None, temperature: float = 1.0, stream=None) -> None:
    """``dlogits`` (may be ``logits``): the gradient of scale * sum of dloss *
    loss with respect to ``logits``, the whole vocabulary's or (with ``first``
    and ``vocab``, also of the first and last one) a shard's.  ``stats`` is
    ``distill``'s or ``distill_join``'s; ``dloss`` [tokens] (float32) may be None
    for all 1."""
    if first != 0 and vocab is None:  # the teacher's distribution is over all of its choices
        raise ValueError("distill_backward: a shard (first) needs the whole vocabulary's size (vocab)")
    ld, ld_d = _matrix(logits, "distill_backward: logits"), _matrix(dlogits, "distill_backward: dlogits")
    dt = _float(logits, "distill_backward: logits")
    _pair(logits, dlogits, "distill_backward: logits and dlogits")
    t, w = logits.shape
    if dlogits.shape != logits.shape:
        raise ValueError("distill_backward: dlogits must have the shape of logits")
    h = _teacher(ids, teacher, t, w if vocab is None else vocab, temperature, "distill_backward")
    _packed(stats, (t, 2), torch.float32, "distill_backward: stats")
    if dloss is not None:
        _packed(dloss, (t,), torch.float32, "distill_backward: dloss")
    on = _device("distill_backward", logits, ids, teacher, stats, dloss, dlogits)
    snac_distill_backward(h, logits, ld, first, w, stats, dloss, scale, t, dt, dlogits, ld_d, _stream(stream, on))
