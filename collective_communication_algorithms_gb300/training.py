"""Training operators on torch CUDA tensors: the embedding lookup, the norms
and the gate at a block's boundary and the distillation loss, each with its
gradient (include/hc.h, "Training operators").  They run on their tensors' GPU,
whichever is current.

Every operator comes as a function that runs once and returns its outputs,
and as bind_*, which returns a BoundCall with `.outputs` (a dict of tensors)
that repeats the call on the same buffers: bind once, call every step.  A
bound call keeps its tensors alive, and runs on the stream current when it was
bound (or `stream`).  Outputs and scratch that are not passed are allocated by
bind_*.  Matrices need unit column stride; rows may be strided.  Nothing here
computes: the work happens in libhc's kernels.
"""
import functools

from . import _binding as B

__all__ = ["embedding", "embedding_grad", "block_norm", "block_norm_grad", "distill", "distill_grad",
           "bind_embedding", "bind_embedding_grad", "bind_block_norm", "bind_block_norm_grad",
           "bind_distill", "bind_distill_grad"]

_FLOATS = {"torch.float32": "float32", "torch.bfloat16": "bfloat16"}
_IDS = {"torch.int32": "int32", "torch.int64": "int64"}


def _dtype(t, table=_FLOATS):
    name = table.get(str(t.dtype))
    if name is None:
        raise TypeError("unsupported dtype %s (%s)" % (t.dtype, ", ".join(table.values())))
    return name


def _check(name, t, shape, dtype=None, device=None, contiguous=False):
    """A CUDA tensor of this shape whose last dimension is dense."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, not %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and str(t.dtype) != str(dtype):
        raise TypeError("%s is %s, not %s" % (name, t.dtype, dtype))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s must have unit column stride" % name)
    return t


def _matrix(t):
    """(pointer, row stride) of a matrix."""
    if t.shape[0] < 2:
        return t.data_ptr(), t.shape[1]
    if t.stride(0) < t.shape[1]:  # expanded, or overlapping rows
        raise ValueError("rows must not overlap (row stride %d of %d columns)" % (t.stride(0), t.shape[1]))
    return t.data_ptr(), t.stride(0)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _new(like, shape, dtype):
    import torch
    return torch.empty(shape, dtype=dtype, device=like.device)


def _scratch(name, args, scratch, like):
    need = B.hc_operator_scratch_bytes(name, args)
    if scratch is None and need:
        import torch
        scratch = _new(like, (need,), torch.uint8)
    if scratch is not None:
        if not scratch.is_cuda or scratch.device != like.device or not scratch.is_contiguous():
            raise ValueError("scratch must be a contiguous tensor on %s" % like.device)
        args.scratch = scratch.data_ptr()
        args.scratch_bytes = scratch.numel() * scratch.element_size()
    return scratch


class _DeviceCall(B.BoundCall):
    """A bound call in a process with several GPUs: the library launches on the
    current one, which has to be that of the tensors and the stream."""

    __slots__ = ("device",)

    def __call__(self):
        import torch
        with torch.cuda.device(self.device):
            super().__call__()


def _bind(name, args, stream, outputs, keep, like):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(like.device)
    elif stream.device != like.device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, like.device))
    if torch.cuda.device_count() > 1:
        call = B.bind_operator(name, args, keep, stream.cuda_stream, _DeviceCall)
        call.device = like.device
    else:
        call = B.bind_operator(name, args, keep, stream.cuda_stream)
    call.outputs = outputs
    return call


def _tensors(kept):
    for k in kept:
        if isinstance(k, (tuple, list)):
            yield from _tensors(k)
        elif isinstance(k, dict):
            yield from _tensors(k.values())
        elif hasattr(k, "record_stream"):
            yield k


def _on_stream(bind):
    """bind_* for a `stream` (a torch stream, or its handle) other than the
    current one.  torch hands freed memory out again in the order of the stream
    that it was allocated on, and the kernels run on another: what the call
    allocates is therefore allocated on the call's stream, and every tensor is
    recorded on the stream that it is a stranger to, so that none is handed out
    while a kernel of the call may still use it."""
    @functools.wraps(bind)
    def run(*args, stream=None, **kw):
        if stream is None:
            return bind(*args, **kw)
        import torch
        first = next(_tensors([args, kw]), None)
        if first is None or not first.is_cuda:
            raise ValueError("stream= is for CUDA tensors")
        device = first.device
        current = torch.cuda.current_stream(device)
        if not hasattr(stream, "cuda_stream"):
            stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                      else torch.cuda.default_stream(device))
        if stream.device == device and stream.cuda_stream == current.cuda_stream:
            return bind(*args, **kw)
        with torch.cuda.stream(stream):
            call = bind(*args, stream=stream, **kw)
        for t in _tensors(call.keep):
            t.record_stream(stream)
        for t in _tensors([call.outputs]):
            t.record_stream(current)
        return call
    return run


@_on_stream
def bind_embedding(table, ids, out=None, scale=1.0, first_id=0, out_dtype=None, *, stream=None):
    """out[t] = scale * table[ids[t] - first_id], zero rows for ids elsewhere;
    `ids` of any shape, `out` (ids.numel(), dim) in out_dtype (the table's)."""
    import torch
    rows, dim = table.shape
    _check("table", table, (rows, dim))
    _check("ids", ids, ids.shape, device=table.device, contiguous=True)
    tokens = ids.numel()
    if out is None:
        out = _new(table, (tokens, dim), out_dtype or table.dtype)
    _check("out", out, (tokens, dim), dtype=out_dtype, device=table.device)
    p, ps = _matrix(table)
    o, os_ = _matrix(out)
    args = B.operator_args("hc_embedding", table=p, ids=_ptr(ids), out=o, tokens=tokens, rows=rows, dim=dim,
                           table_stride=ps, out_stride=os_, table_dtype=_dtype(table), out_dtype=_dtype(out),
                           id_type=_dtype(ids, _IDS), scale=scale, first_id=first_id)
    return _bind("hc_embedding", args, stream, {"out": out}, (table, ids, out), table)


@_on_stream
def bind_embedding_grad(grad_out, ids, grad_table, scale=1.0, first_id=0, padding_id=-1, accumulate=False,
                        scratch=None, *, stream=None):
    """grad_table[v] (+)= scale * sum of grad_out[t] over ids[t] == first_id + v
    (ids equal to padding_id left out)."""
    rows, dim = grad_table.shape
    tokens = ids.numel()
    _check("grad_table", grad_table, (rows, dim))
    _check("grad_out", grad_out, (tokens, dim), device=grad_table.device)
    _check("ids", ids, ids.shape, device=grad_table.device, contiguous=True)
    g, gs = _matrix(grad_out)
    p, ps = _matrix(grad_table)
    args = B.operator_args("hc_embedding_grad", grad_out=g, ids=_ptr(ids), grad_table=p, tokens=tokens, rows=rows,
                           dim=dim, grad_out_stride=gs, grad_table_stride=ps, grad_out_dtype=_dtype(grad_out),
                           grad_table_dtype=_dtype(grad_table), id_type=_dtype(ids, _IDS), scale=scale,
                           first_id=first_id, padding_id=padding_id, accumulate=1 if accumulate else 0)
    scratch = _scratch("hc_embedding_grad", args, scratch, grad_table)
    return _bind("hc_embedding_grad", args, stream, {"grad_table": grad_table},
                 (grad_out, ids, grad_table, scratch), grad_table)


def _norm_weights(y, post_weight, gate, pre_weight):
    """Checks the weights; returns (gate rows, dtype name)."""
    tokens, dim = y.shape
    given = [w for w in (post_weight, gate, pre_weight) if w is not None]
    dtype = given[0].dtype if given else None
    for name, w in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if w is not None:
            _check(name, w, (dim,), dtype, y.device, contiguous=True)
    gate_rows = 0
    if gate is not None:
        if gate.dim() != 2 or gate.shape[0] < 1 or tokens % gate.shape[0]:
            raise ValueError("gate must be (rows, %d) with rows dividing %d" % (dim, tokens))
        _check("gate", gate, (gate.shape[0], dim), dtype, y.device, contiguous=True)
        gate_rows = gate.shape[0]
    return gate_rows, _dtype(given[0]) if given else "float32"


@_on_stream
def bind_block_norm(y, x, post_weight=None, gate=None, pre_weight=None, r=None, z=None, post_rstd=None,
                    pre_rstd=None, residual_scale=1.0, eps=1e-6, next_norm=True, *, stream=None):
    """r = residual_scale * x + gate * rmsnorm(y) * post_weight and
    z = rmsnorm(r) * pre_weight, with the reciprocal root mean squares kept for
    the gradient.  r may be x or y, z too, in place; next_norm=False: r alone."""
    import torch
    tokens, dim = y.shape
    _check("y", y, (tokens, dim))
    _check("x", x, (tokens, dim), y.dtype, y.device)
    gate_rows, wdt = _norm_weights(y, post_weight, gate, pre_weight)
    r = _new(y, (tokens, dim), y.dtype) if r is None else r
    post_rstd = _new(y, (tokens,), torch.float32) if post_rstd is None else post_rstd
    _check("r", r, (tokens, dim), y.dtype, y.device)
    _check("post_rstd", post_rstd, (tokens,), torch.float32, y.device, contiguous=True)
    outputs = {"r": r, "post_rstd": post_rstd}
    zp, zs = None, 0
    if next_norm:
        z = _new(y, (tokens, dim), y.dtype) if z is None else z
        pre_rstd = _new(y, (tokens,), torch.float32) if pre_rstd is None else pre_rstd
        _check("z", z, (tokens, dim), y.dtype, y.device)
        _check("pre_rstd", pre_rstd, (tokens,), torch.float32, y.device, contiguous=True)
        outputs.update(z=z, pre_rstd=pre_rstd)
        zp, zs = _matrix(z)
    elif z is not None or pre_rstd is not None:
        raise ValueError("z and pre_rstd belong to the next norm")
    (yp, ys), (xp, xs), (rp, rs) = _matrix(y), _matrix(x), _matrix(r)
    args = B.operator_args("hc_block_norm", y=yp, x=xp, post_weight=_ptr(post_weight), gate=_ptr(gate),
                           pre_weight=_ptr(pre_weight), r=rp, z=zp, post_rstd=_ptr(post_rstd),
                           pre_rstd=_ptr(pre_rstd), tokens=tokens, dim=dim, gate_rows=gate_rows, y_stride=ys,
                           x_stride=xs, r_stride=rs, z_stride=zs, dtype=_dtype(y), weight_dtype=wdt,
                           residual_scale=residual_scale, eps=eps)
    return _bind("hc_block_norm", args, stream, outputs, (y, x, post_weight, gate, pre_weight, outputs), y)


@_on_stream
def bind_block_norm_grad(grad_r, grad_z, y, x, post_rstd, pre_rstd, post_weight=None, gate=None, pre_weight=None,
                         grad_y=None, grad_x=None, grad_post_weight=None, grad_gate=None, grad_pre_weight=None,
                         residual_scale=1.0, scratch=None, *, stream=None):
    """Gradients of y, x and of every weight that is given, from those of r
    and z (None: zeros, not both) and what block_norm kept."""
    import torch
    tokens, dim = y.shape
    _check("y", y, (tokens, dim))
    _check("x", x, (tokens, dim), y.dtype, y.device)
    if grad_r is None and grad_z is None:
        raise ValueError("grad_r or grad_z is needed")
    for name, t in (("grad_r", grad_r), ("grad_z", grad_z)):
        if t is not None:
            _check(name, t, (tokens, dim), y.dtype, y.device)
    _check("post_rstd", post_rstd, (tokens,), torch.float32, y.device, contiguous=True)
    if grad_z is not None:
        _check("pre_rstd", pre_rstd, (tokens,), torch.float32, y.device, contiguous=True)
    gate_rows, wdt = _norm_weights(y, post_weight, gate, pre_weight)
    grad_y = _new(y, (tokens, dim), y.dtype) if grad_y is None else grad_y
    grad_x = _new(y, (tokens, dim), y.dtype) if grad_x is None else grad_x
    outputs = {"grad_y": grad_y, "grad_x": grad_x}
    for name, t in outputs.items():
        _check(name, t, (tokens, dim), y.dtype, y.device)
    for name, w, g in (("grad_post_weight", post_weight, grad_post_weight), ("grad_gate", gate, grad_gate),
                       ("grad_pre_weight", pre_weight, grad_pre_weight)):
        if w is None:
            if g is not None:
                raise ValueError("%s without its weight" % name)
            continue
        g = _new(y, tuple(w.shape), w.dtype) if g is None else g
        outputs[name] = _check(name, g, tuple(w.shape), w.dtype, y.device, contiguous=True)
    kw = {}
    for name, t in (("grad_r", grad_r), ("grad_z", grad_z), ("y", y), ("x", x), ("grad_y", grad_y),
                    ("grad_x", grad_x)):
        kw[name], kw[name + "_stride"] = _matrix(t) if t is not None else (None, 0)
    args = B.operator_args("hc_block_norm_grad", post_weight=_ptr(post_weight), gate=_ptr(gate),
                           pre_weight=_ptr(pre_weight), post_rstd=_ptr(post_rstd),
                           pre_rstd=_ptr(pre_rstd) if grad_z is not None else None,
                           grad_post_weight=_ptr(outputs.get("grad_post_weight")),
                           grad_gate=_ptr(outputs.get("grad_gate")),
                           grad_pre_weight=_ptr(outputs.get("grad_pre_weight")), tokens=tokens, dim=dim,
                           gate_rows=gate_rows, dtype=_dtype(y), weight_dtype=wdt, residual_scale=residual_scale,
                           **kw)
    scratch = _scratch("hc_block_norm_grad", args, scratch, y)
    return _bind("hc_block_norm_grad", args, stream, outputs,
                 (grad_r, grad_z, y, x, post_weight, gate, pre_weight, post_rstd, pre_rstd, scratch, outputs), y)


def _distill_args(name, logits, teacher_logits, teacher_ids, row_weight, loss, stats, grad, temperature, scale):
    import torch
    tokens, vocab = logits.shape
    top = teacher_logits.shape[1]
    _check("logits", logits, (tokens, vocab))
    _check("teacher_logits", teacher_logits, (tokens, top), device=logits.device)
    _check("teacher_ids", teacher_ids, (tokens, top), device=logits.device)
    lp, ls = _matrix(logits)
    tp, ts = _matrix(teacher_logits)
    ip, is_ = _matrix(teacher_ids)
    if ts != is_:
        raise ValueError("teacher_logits and teacher_ids must have the same row stride")
    if row_weight is not None:
        _check("row_weight", row_weight, (tokens,), torch.float32, logits.device, contiguous=True)
    gp, gs = None, 0
    if grad is not None:
        _check("grad", grad, (tokens, vocab), logits.dtype, logits.device)
        gp, gs = _matrix(grad)
    if loss is not None:
        _check("loss", loss, (tokens,), torch.float32, logits.device, contiguous=True)
    if stats is not None:
        _check("stats", stats, (tokens, 2), torch.float32, logits.device, contiguous=True)
    return B.operator_args(name, logits=lp, teacher_logits=tp, teacher_ids=ip, row_weight=_ptr(row_weight),
                           loss=_ptr(loss), stats=_ptr(stats), grad_logits=gp, tokens=tokens, vocab=vocab, top=top,
                           logits_stride=ls, teacher_stride=ts, grad_stride=gs, dtype=_dtype(logits),
                           teacher_dtype=_dtype(teacher_logits), id_type=_dtype(teacher_ids, _IDS),
                           temperature=temperature, scale=scale)


@_on_stream
def bind_distill(logits, teacher_logits, teacher_ids, row_weight=None, loss=None, stats=None, grad=True,
                 temperature=1.0, scale=1.0, *, stream=None):
    """Per-row distillation loss, and with it the gradient of its sum over the
    logits: grad=True (a new tensor), a tensor (`logits` itself: in place), or
    False (the loss and stats alone, for distill_grad later)."""
    import torch
    tokens = logits.shape[0]
    if grad is True:
        grad = _new(logits, tuple(logits.shape), logits.dtype)
    elif grad is False:
        grad = None
    loss = _new(logits, (tokens,), torch.float32) if loss is None else loss
    stats = _new(logits, (tokens, 2), torch.float32) if stats is None else stats
    args = _distill_args("hc_distill", logits, teacher_logits, teacher_ids, row_weight, loss, stats, grad,
                         temperature, scale)
    outputs = {"loss": loss, "stats": stats}
    if grad is not None:
        outputs["grad"] = grad
    return _bind("hc_distill", args, stream, outputs, (logits, teacher_logits, teacher_ids, row_weight, outputs),
                 logits)


@_on_stream
def bind_distill_grad(logits, teacher_logits, teacher_ids, stats, row_weight=None, grad=None, temperature=1.0,
                      scale=1.0, *, stream=None):
    """The gradient alone, from the stats that distill kept; row_weight is
    then the gradient of the rows' losses."""
    grad = _new(logits, tuple(logits.shape), logits.dtype) if grad is None else grad
    args = _distill_args("hc_distill_grad", logits, teacher_logits, teacher_ids, row_weight, None, stats, grad,
                         temperature, scale)
    return _bind("hc_distill_grad", args, stream, {"grad": grad},
                 (logits, teacher_logits, teacher_ids, row_weight, stats, grad), logits)


def _once(bind, doc):
    def run(*args, **kw):
        call = bind(*args, **kw)
        call()
        return call.outputs
    run.__name__ = bind.__name__[len("bind_"):]
    run.__doc__ = doc + "\n\n    " + bind.__doc__
    return run


embedding = _once(bind_embedding, "One embedding lookup; returns {out}.")
embedding_grad = _once(bind_embedding_grad, "One gradient of the lookup; returns {grad_table}.")
block_norm = _once(bind_block_norm, "One block boundary; returns {r, post_rstd, z, pre_rstd}.")
block_norm_grad = _once(bind_block_norm_grad, "One gradient of the block boundary; returns {grad_y, grad_x, "
                                              "grad_post_weight, grad_gate, grad_pre_weight}.")
distill = _once(bind_distill, "One distillation loss; returns {loss, stats, grad}.")
distill_grad = _once(bind_distill_grad, "One gradient of the distillation loss; returns {grad}.")
