"""Tokens sorted by expert and back, over torch tensors: the plan of a
router's choices, rows handed out to the experts, their results put together
with the choices' weights, and the gradients of both ways.

A training step, with ``experts`` and ``weights`` a token's choices:

    order, place, ends = expert_plan(experts, groups)
    rows = dispatch(x, place, ends)
    ...                                    products grouped by ``ends``
    out = combine(y, place, weights, residual)

    dy, dweights = combine_backward(dout, y, place, weights, ends)
    ...                                    their gradients
    dx = combine(drows, place, residual=dout)

(dout is the gradient of the residual, so the last line adds it to that of x
where both are the same tensor.)  Nothing here waits for the device.  As in
experts.py, calls only read shapes, strides and pointers, allocate what is not
passed in, and forward to the C entry points of include/gemm.h.
"""
from __future__ import annotations

from ._lib import (
    gemm_combine, gemm_combine_backward, gemm_dispatch, gemm_expert_plan, gemm_expert_plan_workspace_size)
from .experts import _call, _check, _common, _device, _elsewhere, _float_type, _ld, _new


def _check_place(place, device: int):
    """(tokens, top) of a plan's places."""
    import torch
    _check(place, "place", device, dtype=torch.int32)
    if not place.is_contiguous():
        raise ValueError("place must be contiguous")
    return place.shape


def _last_end(ends, device: int) -> int:
    """Address of the row that the last group ends before."""
    import torch
    _check(ends, "ends", device, dtype=torch.int32, dim=1)
    groups = ends.shape[0]
    if groups < 1 or (groups > 1 and ends.stride(0) != 1):
        raise ValueError("ends must be contiguous, of one group at least")
    return ends.data_ptr() + 4 * (groups - 1)


def _check_weights(weights, device: int, shape) -> int:
    """Stride of the weights' rows."""
    import torch
    _check(weights, "weights", device, shape, torch.float32)
    return max(_ld(weights, "weights"), shape[1])


def expert_plan(experts, groups: int, stream=None):
    """(order, place, ends) of a router's choices.

    ``experts`` (tokens x top, int64 as topk gives them, or int32) holds each
    token's groups; a number outside 0 .. groups - 1 gives its choice no row.
    ``ends`` (int32, groups) holds the row that each group ends before, as
    ``grouped_gemm`` reads it; ``place`` (int32, tokens x top) the row of each
    choice, or -1; ``order`` (int32, tokens * top) the choice, token * top + k,
    of each row, or -1 past the last end.  A group's rows are in the order of
    their choices."""
    import torch
    if stream is None and experts.is_cuda:
        got = _common("expert_plan", experts, groups)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, experts, expert_plan, experts, groups)
        if got is not None:
            return got
    if experts.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"experts must be int32 or int64 (got {experts.dtype})")
    device = _device(experts, "experts")
    _check(experts, "experts", device)
    tokens, top = experts.shape
    groups = int(groups)
    if top < 1 or groups < 1:
        raise ValueError(f"a token has one choice at least, of one group at least (got {top}, {groups})")

    def new(*shape):
        return torch.empty(shape, dtype=torch.int32, device=experts.device)

    order, place, ends = new(tokens * top), new(tokens, top), new(groups)
    need = gemm_expert_plan_workspace_size(tokens, top, groups)
    ws = new(need // 4) if need else None
    _call("expert_plan", device, gemm_expert_plan, 8 if experts.dtype is torch.int64 else 4, tokens, top, groups,
          experts.data_ptr(), max(_ld(experts, "experts"), top), order.data_ptr(), place.data_ptr(), ends.data_ptr(),
          ws.data_ptr() if need else 0, need)
    return order, place, ends


def dispatch(x, place, ends, scales=None, out=None, out_scales=None, stream=None):
    """out[place[t, k]] = x[t] for every choice that has a row: ``out``, or (out, out_scales).

    ``x`` (tokens x N) is float32, bfloat16, float8_e4m3fn or int8; ``scales``
    (float32, tokens or tokens x blocks) goes along with quantised rows.
    ``out`` has tokens * top rows, or as many as the tensor passed in; rows from
    the last of ``ends`` on become zero, others that no place names are left
    as they were.  The gradient of x is ``combine(drows, place)``."""
    import torch
    if out is None and out_scales is None and stream is None and x.is_cuda:
        got = _common("dispatch", x, place, ends, scales)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, x, dispatch, x, place, ends, scales, out, out_scales)
        if got is not None:
            return got
    if x.dtype not in (torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int8):
        raise TypeError(f"x must be float32, bfloat16, float8_e4m3fn or int8 (got {x.dtype})")
    device = _device(x, "x")
    _check(x, "x", device)
    tokens, top = _check_place(place, device)
    if x.shape[0] != tokens:
        raise ValueError(f"x and place differ in tokens: {tuple(x.shape)}, {tuple(place.shape)}")
    last = _last_end(ends, device)
    N = x.shape[1]
    if out is None:
        out, ldo = _new(tokens * top, N, x.dtype, x.device, 16 if x.itemsize == 1 else 1)
    else:
        _check(out, "out", device, dtype=x.dtype)
        if out.shape[1] != N:
            raise ValueError(f"out must have {N} columns, got shape {tuple(out.shape)}")
        ldo = _ld(out, "out")
    rows, cols, lds, ldos = out.shape[0], 0, 0, 0
    if scales is not None:
        if scales.dim() not in (1, 2) or scales.shape[0] != tokens:
            raise ValueError(f"scales must have shape ({tokens},) or ({tokens}, blocks), got {tuple(scales.shape)}")
        _check(scales, "scales", device, scales.shape, torch.float32)
        shape = (rows, *scales.shape[1:])
        if out_scales is None:
            out_scales = torch.empty(shape, dtype=torch.float32, device=x.device)
        _check(out_scales, "out_scales", device, shape, torch.float32)
        cols = scales.shape[1] if scales.dim() == 2 else 1
        lds, ldos = (_ld(t.view(-1, 1) if t.dim() == 1 else t, what)
                     for t, what in ((scales, "scales"), (out_scales, "out_scales")))
    elif out_scales is not None:
        raise ValueError("out_scales go with scales")
    _call("dispatch", device, gemm_dispatch, x.itemsize, tokens, top, N, x.data_ptr(), _ld(x, "x"), place.data_ptr(), last,
          rows, out.data_ptr(), ldo, cols, scales.data_ptr() if cols else 0, lds, out_scales.data_ptr() if cols else 0,
          ldos)
    return out if scales is None else (out, out_scales)


def combine(rows, place, weights=None, residual=None, out=None, stream=None):
    """out[t] = residual[t] + sum over k of weights[t, k] * rows[place[t, k]].

    ``rows`` and ``residual`` (tokens x N) share a type, float32 or bfloat16,
    which ``out`` has too; sums are float32.  ``weights`` is float32, tokens x
    top (None: all 1).  Choices without a row add nothing.  ``out`` may be
    passed as residual."""
    if out is None and stream is None and rows.is_cuda:
        got = _common("combine", rows, place, weights, residual)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, rows, combine, rows, place, weights, residual, out)
        if got is not None:
            return got
    dt = _float_type(rows, "rows")
    device = _device(rows, "rows")
    _check(rows, "rows", device)
    tokens, top = _check_place(place, device)
    n_rows, N = rows.shape
    w_ptr = r_ptr = ldw = ld_res = 0
    if weights is not None:
        ldw, w_ptr = _check_weights(weights, device, (tokens, top)), weights.data_ptr()
    if residual is not None:
        _check(residual, "residual", device, (tokens, N), rows.dtype)
        r_ptr, ld_res = residual.data_ptr(), _ld(residual, "residual")
    if out is None:
        out, ldo = _new(tokens, N, rows.dtype, rows.device)
    else:
        _check(out, "out", device, (tokens, N), rows.dtype)
        ldo = _ld(out, "out")
    _call("combine", device, gemm_combine, dt, tokens, top, N, rows.data_ptr(), _ld(rows, "rows"), n_rows,
          place.data_ptr(), w_ptr, ldw, r_ptr, ld_res, out.data_ptr(), ldo)
    return out


def combine_backward(dout, rows, place, weights, ends, drows=None, want_dweights: bool = True, stream=None):
    """(drows, dweights) of ``combine``, from the gradient ``dout`` of its output.

    drows[place[t, k]] = weights[t, k] * dout[t], in dout's type; its rows from
    the last of ``ends`` on become zero (it may be passed as rows).  dweights
    (float32, tokens x top; None if it is not wanted) is the product of dout[t]
    with each of its rows, 0 for choices without one.  The residual's gradient
    is dout."""
    import torch
    if drows is None and want_dweights and stream is None and dout.is_cuda:
        got = _common("combine_backward", dout, rows, place, weights, ends)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, dout, combine_backward, dout, rows, place, weights, ends, drows, want_dweights)
        if got is not None:
            return got
    dt = _float_type(dout, "dout")
    device = _device(dout, "dout")
    _check(dout, "dout", device)
    tokens, top = _check_place(place, device)
    if dout.shape[0] != tokens:
        raise ValueError(f"dout and place differ in tokens: {tuple(dout.shape)}, {tuple(place.shape)}")
    N = dout.shape[1]
    _check(rows, "rows", device, dtype=dout.dtype)
    if rows.shape[1] != N:
        raise ValueError(f"rows must have {N} columns, got shape {tuple(rows.shape)}")
    last = _last_end(ends, device)
    ldw = _check_weights(weights, device, (tokens, top))
    if drows is None:
        drows, lddr = _new(rows.shape[0], N, dout.dtype, dout.device)
    else:
        _check(drows, "drows", device, rows.shape, dout.dtype)
        lddr = _ld(drows, "drows")
    dweights = torch.empty((tokens, top), dtype=torch.float32, device=dout.device) if want_dweights else None
    _call("combine_backward", device, gemm_combine_backward, dt, tokens, top, N, dout.data_ptr(), _ld(dout, "dout"),
          rows.data_ptr(), _ld(rows, "rows"), rows.shape[0], place.data_ptr(), last, weights.data_ptr(), ldw,
          drows.data_ptr(), lddr, dweights.data_ptr() if want_dweights else 0, top)
    return drows, dweights
