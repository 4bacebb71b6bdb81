"""The routed experts' operators, and dropout (C ABI in ``include/route_experts.h``).

What a layer runs between the route step's ids and weights and the residual
stream.  Argument marshalling only, as in ``layer.py``, whose plans' methods
(``saved_bytes``, ``new_saved``, ``status``, ``close``) these have too.

* ``DispatchPlan`` -- ``dispatch_sort`` (the pairs of rows and experts sorted by
  expert), ``dispatch_gather`` (rows copied to their sorted places) and
  ``dispatch_combine`` (the experts' results back as weighted sums), with
  ``dispatch_gather_backward`` and ``dispatch_combine_backward``;
* ``ExpertsPlan`` -- ``experts_forward`` / ``experts_backward``: every expert's
  gated block on its run of the sorted rows;
* ``DropoutPlan`` -- ``dropout_forward`` / ``dropout_backward``, from a
  counter-based generator, added to a residual.

The rows of a call are those of its ``x`` (``ids``, ``place``, backward:
``dout``); sorted rows are as many as the tensor has.
"""

from __future__ import annotations

import ctypes

import latent_projection_top_gb300 as _route

from . import layer as _layer
from .layer import (
    _MAT, _act_code, _c_int, _call, _i32, _i64, _LayerPlan, _mat, _opt_mat, _refuse, _rows,
    _saved, _stream, _taken, _type_code, _vp)

MAX_EXPERTS = 1024
MAX_TOPK = 32
EXPERTS_MAX_ROWS = 1048576

# Every symbol include/route_experts.h declares (checked by the CPU tests).
EXPORTS = (
    "route_dispatch_prepare", "route_dispatch_sort", "route_dispatch_gather",
    "route_dispatch_gather_backward", "route_dispatch_combine", "route_dispatch_combine_backward",
    "route_experts_prepare", "route_experts_forward", "route_experts_backward",
    "route_dropout_prepare", "route_dropout_forward", "route_dropout_backward",
)

_u64, _f64 = ctypes.c_uint64, ctypes.c_double
_STACK = [_vp, _i64, _i64]  # the experts' matrices: pointer, row stride, experts' stride


def declare(L) -> None:
    """Argument types of these entry points of the loaded library."""
    out = ctypes.POINTER(_vp)
    L.route_dispatch_prepare.argtypes = [_i32] * 7 + [out]
    L.route_experts_prepare.argtypes = [_i32] * 9 + [out]
    L.route_dropout_prepare.argtypes = [_i32] * 4 + [out]
    head = [_vp, _i32]
    L.route_dispatch_sort.argtypes = head + _MAT + [_vp] * 4
    L.route_dispatch_gather.argtypes = head + _MAT + [_vp, _i32] + _MAT + [_vp]
    L.route_dispatch_gather_backward.argtypes = head + _MAT + [_i32, _vp] + _MAT + [_vp]
    L.route_dispatch_combine.argtypes = head + _MAT + [_i32, _vp, _vp] + _MAT * 2 + [_vp]
    L.route_dispatch_combine_backward.argtypes = head + _MAT * 2 + [_i32, _vp, _vp] + _MAT + [_vp, _vp]
    L.route_experts_forward.argtypes = head + _MAT + [_vp] + _STACK * 3 + _MAT + [_vp, _vp]
    L.route_experts_backward.argtypes = (head + _MAT * 2 + [_vp] + _STACK * 3 + [_vp] + _MAT
                                         + _STACK * 3 + [_vp])
    L.route_dropout_forward.argtypes = head + _MAT + [_f64, _u64, _u64, _vp] + _MAT * 2 + [_vp]
    L.route_dropout_backward.argtypes = head + _MAT + [_f64, _u64, _u64, _vp] + _MAT + [_vp]
    for name in EXPORTS:
        getattr(L, name).restype = _i32


class DispatchPlan(_LayerPlan):
    """Sort, gather and combine for up to `rows` token rows of `dim` values
    (BF16, FP16 or FP32) with `topk` expert ids each; the experts here are
    ``first .. first + experts - 1``."""

    def __init__(self, rows: int, dim: int, dtype, experts: int = _route.N_EXPERTS,
                 topk: int = _route.TOPK, first: int = 0, device: int = 0):
        super().__init__("route_dispatch_prepare", rows, dtype, device, _c_int(dim),
                         _type_code(dtype), _c_int(experts), _c_int(first), _c_int(topk),
                         widths=(int(dim), 0, 0), routed=(int(experts), int(topk)))
        self.dim, self.experts, self.topk, self.first = int(dim), int(experts), int(topk), int(first)


class ExpertsPlan(_LayerPlan):
    """``(act(x W_gate[e]) * (x W_up[e])) W_down[e]`` for the rows of each of
    `experts` experts, up to `rows` sorted rows in all; W_gate and W_up
    ``[experts, k, f]``, W_down ``[experts, f, n]``."""

    def __init__(self, rows: int, k: int, f: int, n: int, experts: int, dtype, act: str = "silu",
                 train: bool = False, device: int = 0):
        super().__init__("route_experts_prepare", rows, dtype, device, _c_int(k), _c_int(f), _c_int(n),
                         _c_int(experts), _type_code(dtype), _act_code(act), int(train),
                         widths=(int(k), int(f), int(n)), routed=(int(experts), 0))
        self.k, self.f, self.n, self.experts = int(k), int(f), int(n), int(experts)
        self.act, self.train = act, bool(train)


class DropoutPlan(_LayerPlan):
    """Dropout of up to `rows` rows of `dim` values (BF16, FP16 or FP32)."""

    def __init__(self, rows: int, dim: int, dtype, device: int = 0):
        super().__init__("route_dropout_prepare", rows, dtype, device, _c_int(dim), _type_code(dtype),
                         widths=(int(dim), 0, 0))
        self.dim = int(dim)

    def draws(self, rows: int | None = None) -> int:
        """How far apart the offsets of two calls of `rows` rows are so that no
        lot is drawn twice."""
        return max(0, self.rows if rows is None else int(rows)) * ((self.dim + 7) // 8)


# ---- marshalling ------------------------------------------------------------

_INT32 = _FP32 = None


def _types():
    global _INT32, _FP32
    import torch
    _INT32, _FP32 = torch.int32, torch.float32


def _ints(t, name, shape, device, dtype=None):
    """Pointer of a contiguous array of int32 (or `dtype`)."""
    if _INT32 is None:
        _types()
    dtype = _INT32 if dtype is None else dtype
    try:
        if (t.dtype is dtype and t.get_device() == device and t.shape == shape
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse_array(t, name, shape, dtype, device)


def _refuse_array(t, name, shape, dtype, device):
    import torch
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == device and t.dtype == dtype
            and tuple(t.shape) == tuple(shape)):
        raise ValueError(f"{name} must be contiguous")
    _refuse(t, name, shape, dtype, device)


def _opt_ints(t, name, shape, device, dtype=None):
    return None if t is None else _ints(t, name, shape, device, dtype)


def _weights(t, name, shape, device):
    if _FP32 is None:
        _types()
    return None if t is None else _ints(t, name, shape, device, _FP32)


def _stack(t, name, experts, rows, cols, dtype, device):
    """(pointer, row stride, experts' stride) of [experts, rows, cols]."""
    try:
        if t.dtype is dtype and t.get_device() == device and t.shape == (experts, rows, cols):
            es, ld, unit = t.stride()
            if unit == 1 or cols == 1:
                return t.data_ptr(), ld, es
    except (AttributeError, ValueError):
        pass
    _refuse(t, name, (experts, rows, cols), dtype, device)


def _opt_stack(t, *args):
    return (None, 0, 0) if t is None else _stack(t, *args)


def _c_u64(v, name) -> int:
    v = int(v)
    if not 0 <= v < 2 ** 64:
        raise ValueError(f"{name} {v} does not fit 64 bits without a sign")
    return v


def _step(t, device):
    if t is None:
        return None
    import torch
    return _ints(t, "step", (1,), device, torch.int64)


# ---- the C entry points -------------------------------------------------------

def dispatch_sort(plan: DispatchPlan, ids, offsets, place, source=None, stream=None) -> None:
    """`ids` [rows, topk] int32: `offsets` [experts + 1] receives where each
    expert's run begins, `place` [rows, topk] each pair's place (-1: not here),
    `source` [rows * topk] the pair at each place."""
    if stream is None and plan._plain is not None and _taken(_layer._short.dispatch_sort(
            plan._plain, ids, offsets, place, source, _layer._current_stream(plan.device))):
        return
    if _INT32 is None:
        _types()
    R, dev = _rows(ids, "ids"), plan.device
    _call("route_dispatch_sort", plan, R, *_mat(ids, "ids", R, plan.topk, _INT32, dev),
          _ints(offsets, "offsets", (plan.experts + 1,), dev),
          _ints(place, "place", (R, plan.topk), dev),
          _opt_ints(source, "source", (R * plan.topk,), dev), _stream(stream, dev))


def dispatch_gather(plan: DispatchPlan, x, place, out, stream=None) -> None:
    """``out[place[r, j]] = x[r]``."""
    if stream is None and plan._plain is not None and _taken(_layer._short.dispatch_gather(
            plan._plain, x, place, out, _layer._current_stream(plan.device))):
        return
    R, P, d, dev, dt = _rows(x, "x"), _rows(out, "out"), plan.dim, plan.device, plan.dtype
    _call("route_dispatch_gather", plan, R, *_mat(x, "x", R, d, dt, dev),
          _ints(place, "place", (R, plan.topk), dev), _c_int(P), *_mat(out, "out", P, d, dt, dev),
          _stream(stream, dev))


def dispatch_gather_backward(plan: DispatchPlan, dout, place, dx, stream=None) -> None:
    """``dx[r] = sum over j of dout[place[r, j]]``."""
    if stream is None and plan._plain is not None and _taken(_layer._short.dispatch_gather_backward(
            plan._plain, dout, place, dx, _layer._current_stream(plan.device))):
        return
    R, P, d, dev, dt = _rows(dx, "dx"), _rows(dout, "dout"), plan.dim, plan.device, plan.dtype
    _call("route_dispatch_gather_backward", plan, R, *_mat(dout, "dout", P, d, dt, dev), _c_int(P),
          _ints(place, "place", (R, plan.topk), dev), *_mat(dx, "dx", R, d, dt, dev),
          _stream(stream, dev))


def dispatch_combine(plan: DispatchPlan, y, place, weights, out, residual=None, stream=None) -> None:
    """``out[r] = sum over j of weights[r, j] y[place[r, j]] + residual[r]``;
    weights [rows, topk] FP32 may be None (1)."""
    if stream is None and plan._plain is not None and _taken(_layer._short.dispatch_combine(
            plan._plain, y, place, weights, out, residual, _layer._current_stream(plan.device))):
        return
    R, P, d, dev, dt = _rows(out, "out"), _rows(y, "y"), plan.dim, plan.device, plan.dtype
    _call("route_dispatch_combine", plan, R, *_mat(y, "y", P, d, dt, dev), _c_int(P),
          _ints(place, "place", (R, plan.topk), dev),
          _weights(weights, "weights", (R, plan.topk), dev),
          *_opt_mat(residual, "residual", R, d, dt, dev), *_mat(out, "out", R, d, dt, dev),
          _stream(stream, dev))


def dispatch_combine_backward(plan: DispatchPlan, dout, y, place, weights, dy=None, dweights=None,
                              stream=None) -> None:
    """``dy[place[r, j]] = weights[r, j] dout[r]``, ``dweights[r, j] =
    <dout[r], y[place[r, j]]>``.  y may be None without dweights."""
    if stream is None and plan._plain is not None and _taken(_layer._short.dispatch_combine_backward(
            plan._plain, dout, y, place, weights, dy, dweights, _layer._current_stream(plan.device))):
        return
    R, d, dev, dt = _rows(dout, "dout"), plan.dim, plan.device, plan.dtype
    P = _rows(y, "y") if y is not None else _rows(dy, "dy") if dy is not None else 0
    if dweights is not None and y is None:
        raise TypeError("y must be a 2-D torch.Tensor")
    _call("route_dispatch_combine_backward", plan, R, *_mat(dout, "dout", R, d, dt, dev),
          *_opt_mat(y, "y", P, d, dt, dev), _c_int(P), _ints(place, "place", (R, plan.topk), dev),
          _weights(weights, "weights", (R, plan.topk), dev), *_opt_mat(dy, "dy", P, d, dt, dev),
          _weights(dweights, "dweights", (R, plan.topk), dev), _stream(stream, dev))


def experts_forward(plan: ExpertsPlan, x, offsets, W_gate, W_up, W_down, out, saved=None,
                    stream=None) -> None:
    """`x` [rows, k] sorted by expert, `offsets` [experts + 1] int32: rows that
    are nobody's are not written in `out` [rows, n]."""
    if stream is None and plan._plain is not None and _taken(_layer._short.experts_forward(
            plan._plain, x, offsets, W_gate, W_up, W_down, out, saved, _layer._current_stream(plan.device))):
        return
    R, k, f, n, dev, dt = _rows(x, "x"), plan.k, plan.f, plan.n, plan.device, plan.dtype
    E = plan.experts
    _call("route_experts_forward", plan, R, *_mat(x, "x", R, k, dt, dev),
          _ints(offsets, "offsets", (E + 1,), dev), *_stack(W_gate, "W_gate", E, k, f, dt, dev),
          *_stack(W_up, "W_up", E, k, f, dt, dev), *_stack(W_down, "W_down", E, f, n, dt, dev),
          *_mat(out, "out", R, n, dt, dev), _saved(plan, saved, R), _stream(stream, dev))


def experts_backward(plan: ExpertsPlan, dout, x, offsets, W_gate, W_up, W_down, saved, dx=None,
                     dW_gate=None, dW_up=None, dW_down=None, stream=None) -> None:
    """Any of the gradients; those of an expert's weights without rows are 0."""
    if stream is None and plan._plain is not None and _taken(_layer._short.experts_backward(
            plan._plain, dout, x, offsets, W_gate, W_up, W_down, saved, dx, dW_gate, dW_up, dW_down, _layer._current_stream(plan.device))):
        return
    R, k, f, n, dev, dt = _rows(dout, "dout"), plan.k, plan.f, plan.n, plan.device, plan.dtype
    E = plan.experts
    _call("route_experts_backward", plan, R, *_mat(dout, "dout", R, n, dt, dev),
          *_opt_mat(x, "x", R, k, dt, dev), _ints(offsets, "offsets", (E + 1,), dev),
          *_stack(W_gate, "W_gate", E, k, f, dt, dev), *_stack(W_up, "W_up", E, k, f, dt, dev),
          *_stack(W_down, "W_down", E, f, n, dt, dev), _saved(plan, saved, R),
          *_opt_mat(dx, "dx", R, k, dt, dev), *_opt_stack(dW_gate, "dW_gate", E, k, f, dt, dev),
          *_opt_stack(dW_up, "dW_up", E, k, f, dt, dev),
          *_opt_stack(dW_down, "dW_down", E, f, n, dt, dev), _stream(stream, dev))


def dropout_forward(plan: DropoutPlan, x, p: float, seed: int, out, offset: int = 0, residual=None,
                    step=None, stream=None) -> None:
    """``out = keep * x / (1 - p) + residual``.  The lots are a function of
    `seed`, `offset` and the place in the matrix; calls whose offsets are
    ``plan.draws(rows)`` apart have lots of their own.  `step`, an int64 tensor
    of one value on the device, is added to the offset when the kernel runs
    (for captured calls)."""
    if stream is None and plan._plain is not None and _taken(_layer._short.dropout_forward(
            plan._plain, x, p, seed, out, offset, residual, step, _layer._current_stream(plan.device))):
        return
    R, d, dev, dt = _rows(x, "x"), plan.dim, plan.device, plan.dtype
    _call("route_dropout_forward", plan, R, *_mat(x, "x", R, d, dt, dev), p, _c_u64(seed, "seed"),
          _c_u64(offset, "offset"), _step(step, dev), *_opt_mat(residual, "residual", R, d, dt, dev),
          *_mat(out, "out", R, d, dt, dev), _stream(stream, dev))


def dropout_backward(plan: DropoutPlan, dout, p: float, seed: int, dx, offset: int = 0, step=None,
                     stream=None) -> None:
    """``dx = keep * dout / (1 - p)`` with the lots of the forward call of the
    same seed, offset and step."""
    if stream is None and plan._plain is not None and _taken(_layer._short.dropout_backward(
            plan._plain, dout, p, seed, dx, offset, step, _layer._current_stream(plan.device))):
        return
    R, d, dev, dt = _rows(dout, "dout"), plan.dim, plan.device, plan.dtype
    _call("route_dropout_backward", plan, R, *_mat(dout, "dout", R, d, dt, dev), p,
          _c_u64(seed, "seed"), _c_u64(offset, "offset"), _step(step, dev),
          *_mat(dx, "dx", R, d, dt, dev), _stream(stream, dev))
