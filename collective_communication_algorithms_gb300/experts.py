"""Operators of an expert layer on torch CUDA tensors: the plan that groups a
batch's tokens by expert, the products of each group with its expert's weight
and the weighted sum back to the tokens, with their gradients (include/hc.h,
"Expert layer").  Functions, bind_* and bound calls as in training.py.

The rows between the plan and the sum are the assignments (token, choice)
sorted by expert.  hc.embedding(table=x, ids=plan["tokens"]) gathers them, and
expert_combine without weights is the gradient of that gather.  Outputs that
are not passed begin as zeros where rows of no expert keep what they hold.
"""
from . import _binding as B
from .training import _IDS, _bind, _check, _dtype, _matrix, _new, _on_stream, _once, _ptr, _scratch

__all__ = ["expert_plan", "expert_matmul", "expert_matmul_grad", "expert_combine", "expert_combine_grad",
           "bind_expert_plan", "bind_expert_matmul", "bind_expert_matmul_grad", "bind_expert_combine",
           "bind_expert_combine_grad"]


def _zeros(like, shape, dtype):
    import torch
    return torch.zeros(shape, dtype=dtype, device=like.device)


def _check_weight(name, w, shape, dtype, device):
    if not w.is_cuda or w.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    if tuple(w.shape) != tuple(shape):
        raise ValueError("%s has shape %s, not %s" % (name, tuple(w.shape), tuple(shape)))
    if dtype is not None and w.dtype != dtype:
        raise TypeError("%s is %s, not %s" % (name, w.dtype, dtype))


def _rows_of(w, layout):
    """(rows, columns, row stride, column stride) of an expert's weight in a layout."""
    row, col = (1, 2) if layout == "out_in" else (2, 1)
    return w.shape[row], w.shape[col], w.stride(row), w.stride(col)


def _layout(**weights):
    """The layout that all of these have: experts x out x in ("out_in"), or the
    transposed view of experts x in x out ("in_out").  With one input or one
    output a weight may have both."""
    able = {}
    for name, w in weights.items():
        able[name] = [k for k in B.LAYOUTS for rows, cols, stride, unit in [_rows_of(w, k)]
                      if (cols == 1 or unit == 1) and (rows == 1 or stride >= cols)]
        if not able[name]:
            raise ValueError("%s must have unit stride along its inputs or its outputs, and rows that do not overlap" % name)
    common = [k for k in B.LAYOUTS if all(k in v for v in able.values())]
    if not common:
        raise ValueError("grad_weight must be laid out as weight is (%s)" % able["weight"][0])
    return common[0]


def _experts_weight(name, w, layout):
    """(pointer, row stride, expert stride) of weights in a layout that they have."""
    rows, cols, stride, _ = _rows_of(w, layout)
    if rows == 1:
        stride = cols
    extent = (rows - 1) * stride + cols
    step = w.stride(0) if w.shape[0] > 1 else extent
    if step < extent:
        raise ValueError("%s: experts must not overlap" % name)
    return w.data_ptr(), stride, step


def _offsets(offsets, experts, device):
    import torch
    return _ptr(_check("offsets", offsets, (experts + 1,), torch.int32, device, contiguous=True))


@_on_stream
def bind_expert_plan(expert_ids, num_experts, offsets=None, tokens=None, slots=None, first_expert=0, scratch=None, *,
                     stream=None):
    """For expert_ids (tokens, top): `offsets` (num_experts + 1), the rows of
    each expert; `tokens`, the token of each row (-1 behind the last); `slots`
    (tokens, top), the row of each assignment (-1 for ids outside
    [first_expert, first_expert + num_experts)).  All int32."""
    import torch
    n, top = expert_ids.shape
    _check("expert_ids", expert_ids, (n, top), contiguous=True)
    offsets = _new(expert_ids, (num_experts + 1,), torch.int32) if offsets is None else offsets
    tokens = _new(expert_ids, (n * top,), torch.int32) if tokens is None else tokens
    slots = _new(expert_ids, (n, top), torch.int32) if slots is None else slots
    _check("tokens", tokens, (n * top,), torch.int32, expert_ids.device, contiguous=True)
    _check("slots", slots, (n, top), torch.int32, expert_ids.device, contiguous=True)
    args = B.operator_args("hc_expert_plan", expert_ids=_ptr(expert_ids),
                           offsets=_offsets(offsets, num_experts, expert_ids.device), row_tokens=_ptr(tokens),
                           slots=_ptr(slots), tokens=n, top=top, experts=num_experts,
                           id_type=_dtype(expert_ids, _IDS), first_expert=first_expert)
    scratch = _scratch("hc_expert_plan", args, scratch, expert_ids)
    outputs = {"offsets": offsets, "tokens": tokens, "slots": slots}
    return _bind("hc_expert_plan", args, stream, outputs, (expert_ids, scratch, outputs), expert_ids)


@_on_stream
def bind_expert_matmul(x, weight, offsets, out=None, out_dtype=None, scratch=None, *, stream=None):
    """out[r] = weight[e] @ x[r] for the rows offsets[e] <= r < offsets[e + 1];
    weight (experts, out, in), or the transposed view of (experts, in, out)."""
    rows, inner = x.shape
    experts, outer = weight.shape[0], weight.shape[1]
    _check("x", x, (rows, inner))
    _check_weight("weight", weight, (experts, outer, inner), x.dtype, x.device)
    layout = _layout(weight=weight)
    wp, ws, es = _experts_weight("weight", weight, layout)
    out = _zeros(x, (rows, outer), out_dtype or x.dtype) if out is None else out
    _check("out", out, (rows, outer), out_dtype, x.device)
    (xp, xs), (op, os_) = _matrix(x), _matrix(out)
    args = B.operator_args("hc_expert_matmul", x=xp, weight=wp, offsets=_offsets(offsets, experts, x.device), out=op,
                           rows=rows, experts=experts, in_dim=inner, out_dim=outer, x_stride=xs, weight_stride=ws,
                           expert_stride=es, out_stride=os_, dtype=_dtype(x), out_dtype=_dtype(out),
                           weight_layout=layout)
    scratch = _scratch("hc_expert_matmul", args, scratch, x)
    return _bind("hc_expert_matmul", args, stream, {"out": out}, (x, weight, offsets, out, scratch), x)


@_on_stream
def bind_expert_matmul_grad(grad_out, offsets, x=None, weight=None, grad_x=None, grad_weight=None,
                            grad_weight_dtype=None, accumulate=False, scratch=None, *, stream=None):
    """grad_x[r] = weight[e]^T @ grad_out[r], if weight is given, and
    grad_weight[e] (+)= the sum of grad_out[r] x[r]^T over e's rows, if x is
    (in grad_weight_dtype, x's type; grad_weight's layout is then its own, and
    has to be weight's if that is given too).  What is added to a fp32
    grad_weight of bf16 operands counts as 0 where it is subnormal, as does
    what it holds."""
    rows, outer = grad_out.shape
    experts = offsets.shape[0] - 1
    _check("grad_out", grad_out, (rows, outer))
    if x is None and weight is None:
        raise ValueError("weight (for grad_x) or x (for grad_weight) is needed")
    inner = x.shape[1] if x is not None else weight.shape[2]
    device, kw, outputs, shape = grad_out.device, {}, {}, (experts, outer, inner)
    given = {}
    if weight is not None:
        _check_weight("weight", weight, shape, grad_out.dtype, device)
        given["weight"] = weight
    if x is not None and grad_weight is not None:
        _check_weight("grad_weight", grad_weight, shape, grad_weight_dtype, device)
        given["grad_weight"] = grad_weight
    layout = _layout(**given) if given else "out_in"
    if weight is not None:
        wp, ws, es = _experts_weight("weight", weight, layout)
        grad_x = _zeros(grad_out, (rows, inner), grad_out.dtype) if grad_x is None else grad_x
        _check("grad_x", grad_x, (rows, inner), grad_out.dtype, device)
        gp, gs = _matrix(grad_x)
        kw.update(weight=wp, weight_stride=ws, expert_stride=es, grad_x=gp, grad_x_stride=gs)
        outputs["grad_x"] = grad_x
    elif grad_x is not None:
        raise ValueError("grad_x without weight")
    if x is not None:
        _check("x", x, (rows, inner), grad_out.dtype, device)
        if grad_weight is None:
            if accumulate:
                raise ValueError("accumulate needs grad_weight")
            grad_weight = _new(x, shape if layout == "out_in" else (experts, inner, outer), grad_weight_dtype or x.dtype)
            if layout == "in_out":
                grad_weight = grad_weight.transpose(1, 2)
        gp, gs, ge = _experts_weight("grad_weight", grad_weight, layout)
        xp, xs = _matrix(x)
        kw.update(x=xp, x_stride=xs, grad_weight=gp, grad_weight_stride=gs, grad_expert_stride=ge,
                  grad_weight_dtype=_dtype(grad_weight))
        outputs["grad_weight"] = grad_weight
    else:
        if grad_weight is not None or accumulate:
            raise ValueError("grad_weight without x")
        kw.update(grad_weight_dtype="float32")
    op, os_ = _matrix(grad_out)
    args = B.operator_args("hc_expert_matmul_grad", grad_out=op, offsets=_offsets(offsets, experts, device), rows=rows,
                           experts=experts, in_dim=inner, out_dim=outer, grad_out_stride=os_, dtype=_dtype(grad_out),
                           weight_layout=layout, accumulate=1 if accumulate else 0, **kw)
    scratch = _scratch("hc_expert_matmul_grad", args, scratch, grad_out)
    return _bind("hc_expert_matmul_grad", args, stream, outputs, (grad_out, offsets, x, weight, scratch, outputs),
                 grad_out)


@_on_stream
def bind_expert_combine(y, slots, weights=None, out=None, *, stream=None):
    """out[t] = sum over j of weights[t, j] * y[slots[t, j]] (ones if weights
    is None; slots outside y's rows have no part)."""
    import torch
    rows, dim = y.shape
    tokens, top = slots.shape
    _check("y", y, (rows, dim))
    _check("slots", slots, (tokens, top), torch.int32, y.device, contiguous=True)
    if weights is not None:
        _check("weights", weights, (tokens, top), device=y.device, contiguous=True)
    out = _new(y, (tokens, dim), y.dtype) if out is None else out
    _check("out", out, (tokens, dim), y.dtype, y.device)
    (yp, ys), (op, os_) = _matrix(y), _matrix(out)
    args = B.operator_args("hc_expert_combine", y=yp, slots=_ptr(slots), weights=_ptr(weights), out=op, tokens=tokens,
                           top=top, rows=rows, dim=dim, y_stride=ys, out_stride=os_, dtype=_dtype(y),
                           weight_dtype=_dtype(weights) if weights is not None else "float32")
    return _bind("hc_expert_combine", args, stream, {"out": out}, (y, slots, weights, out), y)


@_on_stream
def bind_expert_combine_grad(grad_out, slots, y=None, weights=None, grad_y=None, grad_weights=None, rows=None,
                             want_grad_y=True, *, stream=None):
    """grad_y[slots[t, j]] = weights[t, j] * grad_out[t] (want_grad_y; other
    rows keep what they hold), and grad_weights[t, j] = <grad_out[t],
    y[slots[t, j]]>, if y and weights are given.  `rows`: those of grad_y if
    neither y nor grad_y says so.  grad_y may be y in place."""
    import torch
    tokens, dim = grad_out.shape
    top = slots.shape[1]
    device = grad_out.device
    _check("grad_out", grad_out, (tokens, dim))
    _check("slots", slots, (tokens, top), torch.int32, device, contiguous=True)
    given = [t.shape[0] for t in (y, grad_y) if t is not None]
    rows = given[0] if given else rows
    if rows is None:
        raise ValueError("y, grad_y or rows is needed")
    kw, outputs = {}, {}
    if weights is not None:
        _check("weights", weights, (tokens, top), device=device, contiguous=True)
        kw.update(weights=_ptr(weights), weight_dtype=_dtype(weights))
    else:
        kw.update(weight_dtype="float32")
    if y is not None:
        _check("y", y, (rows, dim), grad_out.dtype, device)
    if y is not None and weights is not None:
        grad_weights = _new(weights, (tokens, top), weights.dtype) if grad_weights is None else grad_weights
        _check("grad_weights", grad_weights, (tokens, top), weights.dtype, device, contiguous=True)
        yp, ys = _matrix(y)
        kw.update(y=yp, y_stride=ys, grad_weights=_ptr(grad_weights))
        outputs["grad_weights"] = grad_weights
    elif grad_weights is not None:
        raise ValueError("grad_weights without y and weights")
    if want_grad_y:
        grad_y = _zeros(grad_out, (rows, dim), grad_out.dtype) if grad_y is None else grad_y
        _check("grad_y", grad_y, (rows, dim), grad_out.dtype, device)
        gp, gs = _matrix(grad_y)
        kw.update(grad_y=gp, grad_y_stride=gs)
        outputs["grad_y"] = grad_y
    if not outputs:
        raise ValueError("no gradient is asked for")
    op, os_ = _matrix(grad_out)
    args = B.operator_args("hc_expert_combine_grad", grad_out=op, slots=_ptr(slots), tokens=tokens, top=top, rows=rows,
                           dim=dim, grad_out_stride=os_, dtype=_dtype(grad_out), **kw)
    return _bind("hc_expert_combine_grad", args, stream, outputs, (grad_out, slots, y, weights, outputs), grad_out)


expert_plan = _once(bind_expert_plan, "One plan; returns {offsets, tokens, slots}.")
expert_matmul = _once(bind_expert_matmul, "One product of each group; returns {out}.")
expert_matmul_grad = _once(bind_expert_matmul_grad, "Its gradients; returns {grad_x, grad_weight}.")
expert_combine = _once(bind_expert_combine, "One sum back to the tokens; returns {out}.")
expert_combine_grad = _once(bind_expert_combine_grad, "Its gradients; returns {grad_y, grad_weights}.")
