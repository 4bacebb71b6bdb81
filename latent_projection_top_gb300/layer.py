"""The layer operators around the route step (C ABI in ``include/route_layer.h``).

Argument marshalling only, like the route step's binding: tensors are checked
for dtype, shape, stride and device, then their pointers, row strides and the
CUDA stream go to the C entry points of the same names.  Calls whose arguments
are plainly right take a short way where it is built, a compiled module that
makes the same checks (``csrc/layer_call.cpp``: 2 to 5 us less a call); all
others go through the checks here, which raise what is wrong.

* ``norm_forward`` / ``norm_backward`` -- layer norm of token rows;
* ``linear_forward`` / ``linear_backward`` -- ``act(x W + bias) + residual``;
* ``gated_forward`` / ``gated_backward`` -- a gated feed-forward block,
  ``(act(x W_gate) * (x W_up)) W_down + residual``.

Each runs on a plan (``NormPlan``, ``LinearPlan``, ``GatedPlan``) that fixes
the widths, the type and the largest number of rows and owns the scratch
memory; the rows of a call are those of its ``x`` (backward: ``dout``).
Matrices may be views with any row stride (``include/route_layer.h`` states
the alignment that operands need); outputs are written in place.
"""

from __future__ import annotations

import ctypes

import latent_projection_top_gb300 as _route

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")
LAYER_MAX_ROWS = 65536
LAYER_MAX_WIDTH = 65536
NORM_MAX_WIDTH = 16384

# Every symbol include/route_layer.h declares (checked by the CPU tests).
EXPORTS = (
    "route_norm_prepare", "route_linear_prepare", "route_gated_prepare", "route_layer_destroy",
    "route_layer_status", "route_layer_saved_bytes", "route_norm_forward", "route_norm_backward",
    "route_linear_forward", "route_linear_backward", "route_gated_forward",
    "route_gated_backward", "route_layer_test_stall",
)

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
_MAT = [_vp, _i64]  # a matrix: its pointer and row stride


def declare(L) -> None:
    """Argument types of the layer entry points of the loaded library."""
    out = ctypes.POINTER(_vp)
    L.route_norm_prepare.argtypes = [_i32] * 4 + [out]
    L.route_linear_prepare.argtypes = [_i32] * 8 + [out]
    L.route_gated_prepare.argtypes = [_i32] * 8 + [out]
    L.route_layer_destroy.argtypes = [_vp]
    L.route_layer_status.argtypes = [_vp]
    L.route_layer_saved_bytes.argtypes = [_vp, _i32]
    L.route_norm_forward.argtypes = [_vp, _i32] + _MAT + [_vp, _vp, _f32] + _MAT + [_vp, _vp]
    L.route_norm_backward.argtypes = [_vp, _i32] + _MAT * 2 + [_vp, _vp] + _MAT + [_vp, _vp, _vp]
    L.route_linear_forward.argtypes = [_vp, _i32] + _MAT * 2 + [_vp] + _MAT * 2 + [_vp, _vp]
    L.route_linear_backward.argtypes = [_vp, _i32] + _MAT * 3 + [_vp] + _MAT * 2 + [_vp, _vp]
    L.route_gated_forward.argtypes = [_vp, _i32] + _MAT * 6 + [_vp, _vp]
    L.route_gated_backward.argtypes = [_vp, _i32] + _MAT * 5 + [_vp] + _MAT * 4 + [_vp]
    L.route_layer_test_stall.argtypes = [_vp, _i32, ctypes.c_uint64]
    for name in EXPORTS:
        getattr(L, name).restype = _i32
    L.route_layer_saved_bytes.restype = _i64


_TYPES = None
_FP32 = _UINT8 = None  # torch's, once a plan exists


def _type_code(dtype) -> int:
    global _TYPES, _FP32, _UINT8
    if _TYPES is None:
        import torch
        _TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
        _FP32, _UINT8 = torch.float32, torch.uint8
    try:
        return _TYPES[dtype]
    except (KeyError, TypeError):
        raise TypeError(f"dtype {dtype} is not one of {tuple(_TYPES)}") from None


def _c_int(v) -> int:
    """An int as the C ABI takes it; one outside its range stays outside every
    limit there (ctypes would cut it to 32 bits: 2**32 + 4 rows to 4)."""
    return max(-2 ** 31, min(int(v), 2 ** 31 - 1))


def _act_code(act: str) -> int:
    try:
        return ACTIVATIONS.index(act)
    except ValueError:
        raise ValueError(f"activation {act!r} is not one of {ACTIVATIONS}") from None


_short = None
_without = False  # the compiled module could not be loaded


def _short_way():
    """The compiled module, bound to the loaded library; None (and one warning)
    where it is missing or does not load: the calls then go through ctypes."""
    global _short, _without
    if _short is None and not _without:
        import importlib.util
        from importlib.machinery import ExtensionFileLoader

        import torch  # noqa: F401  (the module needs its libraries)

        from . import builder
        L = _route.lib()
        try:
            loader = ExtensionFileLoader("_layer_call", builder.call_module())
            module = importlib.util.module_from_spec(
                importlib.util.spec_from_loader("_layer_call", loader))
            loader.exec_module(module)
        except (ImportError, OSError) as e:
            import warnings
            _without = True
            warnings.warn(f"layer calls go through ctypes, 2 to 5 us more each: {e} "
                          "(latent_projection_top_gb300.build() makes the module)")
            return None
        module.bind(*(ctypes.cast(getattr(L, f"route_{name}"), _vp).value for name in (
            "norm_forward", "norm_backward", "linear_forward", "linear_backward",
            "gated_forward", "gated_backward")))
        _short = module
    return _short


class _LayerPlan:
    """A prepared layer operator; a context manager, or call ``close()``."""

    def __init__(self, prepare: str, rows: int, dtype, device: int, *args, out_dtype=None,
                 widths: tuple):
        self._h = None
        h = ctypes.c_void_p()
        _route._check(getattr(_route.lib(), prepare)(_c_int(rows), *args, _c_int(device),
                                                     ctypes.byref(h)))
        self._h = h
        self._p = h.value  # what the calls pass; None once closed
        self.rows = int(rows)
        self.dtype = dtype
        self.device = int(device)
        # what a training forward call keeps of each row
        self.saved_row = _route._lib.route_layer_saved_bytes(h, 1)
        # the plan as the short way takes it; None once closed, or without the module
        self._plain = None if _short_way() is None else (
            self._p, self.device, _type_code(dtype),
            _type_code(dtype if out_dtype is None else out_dtype), *widths, self.saved_row)

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise _route.RouteError(7, "plan is closed")
        return self._h

    def saved_bytes(self, rows: int | None = None) -> int:
        """Bytes a training forward call of `rows` rows keeps for its backward call."""
        self.handle  # raises: closed
        return self.saved_row * max(0, self.rows if rows is None else int(rows))

    def new_saved(self, rows: int | None = None):
        """A buffer for what a training forward call keeps (None if nothing)."""
        import torch
        n = self.saved_bytes(rows)
        return torch.empty((n,), dtype=torch.uint8, device=f"cuda:{self.device}") if n else None

    def status(self) -> None:
        """Synchronise the device and raise if a kernel of this plan gave up."""
        _route._check(_route.lib().route_layer_status(self.handle))

    def close(self) -> None:
        if self._h is not None and self._h.value:
            _route.lib().route_layer_destroy(self._h)
        self._h = self._p = self._plain = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class NormPlan(_LayerPlan):
    """Layer norm of up to `rows` rows of `dim` values (BF16, FP16 or FP32)."""

    def __init__(self, rows: int, dim: int, dtype, device: int = 0):
        super().__init__("route_norm_prepare", rows, dtype, device, _c_int(dim), _type_code(dtype),
                         widths=(int(dim), 0, 0))
        self.dim = int(dim)


class LinearPlan(_LayerPlan):
    """``act(x W + bias) + residual`` for up to `rows` rows, W ``[k, n]``."""

    def __init__(self, rows: int, k: int, n: int, dtype, act: str = "none", train: bool = False,
                 out_dtype=None, device: int = 0):
        out_dtype = dtype if out_dtype is None else out_dtype
        super().__init__("route_linear_prepare", rows, dtype, device, _c_int(k), _c_int(n),
                         _type_code(dtype), _type_code(out_dtype), _act_code(act), int(train),
                         out_dtype=out_dtype, widths=(int(k), 0, int(n)))
        self.k, self.n, self.act, self.train = int(k), int(n), act, bool(train)
        self.out_dtype = out_dtype


class GatedPlan(_LayerPlan):
    """``(act(x W_gate) * (x W_up)) W_down + residual`` for up to `rows` rows,
    W_gate and W_up ``[k, f]``, W_down ``[f, n]``."""

    def __init__(self, rows: int, k: int, f: int, n: int, dtype, act: str = "silu",
                 train: bool = False, device: int = 0):
        super().__init__("route_gated_prepare", rows, dtype, device, _c_int(k), _c_int(f), _c_int(n),
                         _type_code(dtype), _act_code(act), int(train),
                         widths=(int(k), int(f), int(n)))
        self.k, self.f, self.n, self.act, self.train = int(k), int(f), int(n), act, bool(train)


# ---- marshalling ------------------------------------------------------------

def _refuse(t, name, shape, dtype, device):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda" or t.device.index != device:
        raise ValueError(f"{name} must be on cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}; expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    raise ValueError(f"{name} must have unit stride between columns")


def _mat(t, name, rows, cols, dtype, device):
    """(pointer, row stride) of a matrix with unit stride between columns."""
    try:
        # get_device() is -1 off the GPU
        if t.dtype is dtype and t.get_device() == device and t.shape == (rows, cols):
            ld, unit = t.stride()
            if unit == 1 or cols == 1:
                return t.data_ptr(), ld
    except (AttributeError, ValueError):
        pass
    _refuse(t, name, (rows, cols), dtype, device)


def _opt_mat(t, name, rows, cols, dtype, device):
    return (None, 0) if t is None else _mat(t, name, rows, cols, dtype, device)


def _vec(t, name, n, dtype, device):
    """Pointer of an optional contiguous vector."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.get_device() == device and t.shape == (n,)
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, (n,), dtype, device)


def _stats(t, rows, device, need):
    if t is None and not need:
        return None
    p, ld = _mat(t, "stats", rows, 2, _FP32, device)
    if ld != 2 and rows > 1:
        raise ValueError("stats must be contiguous")
    return p


def _saved(plan, t, rows):
    if t is None:
        return None
    try:
        if (t.dtype is _UINT8 and t.get_device() == plan.device and t.is_contiguous()
                and t.numel() >= rows * plan.saved_row):
            return t.data_ptr()
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
        raise TypeError("saved must be a uint8 tensor (plan.new_saved())")
    if not t.is_cuda or t.get_device() != plan.device or not t.is_contiguous():
        raise ValueError(f"saved must be contiguous and on cuda:{plan.device}")
    raise ValueError(f"saved holds {t.numel()} bytes; {rows} rows need {rows * plan.saved_row}")


def _rows(t, name):
    try:
        return t.shape[0]
    except (AttributeError, IndexError):
        raise TypeError(f"{name} must be a 2-D torch.Tensor") from None


def _stream(stream, device):
    if stream is None:
        return _current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _current_stream(device):
    """torch's current stream as a handle (the first call finds the cheapest
    way to ask: building a Stream object costs as much as a kernel launch)."""
    global _current_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _current_stream = raw if raw is not None else (
        lambda d: torch.cuda.current_stream(d).cuda_stream)
    return torch.cuda.current_stream(device).cuda_stream


def _taken(status) -> bool:
    """Whether the short way took the call; the library's refusal is raised."""
    if status > 0:
        _route._check(status)
    return status == 0


def _call(name, plan, rows, *args):
    """One C entry point; the message of a refusal is its exception's."""
    handle = plan._p
    if handle is None:
        plan.handle  # raises: closed
    status = getattr(_route._lib, name)(handle, _c_int(rows), *args)
    if status:
        _route._check(status)


# ---- the C entry points -------------------------------------------------------

def norm_forward(plan: NormPlan, x, gamma, beta, out, stats=None, eps: float = 1e-5,
                 stream=None) -> None:
    """``out = (x - mean) rstd gamma + beta``; `stats` [rows, 2] FP32 receives
    (mean, rstd).  gamma and beta may be None."""
    if stream is None and plan._plain is not None and _taken(_short.norm_forward(
            plan._plain, x, gamma, beta, out, stats, eps, _current_stream(plan.device))):
        return
    R, d, dev, dt = _rows(x, "x"), plan.dim, plan.device, plan.dtype
    _call("route_norm_forward", plan, R, *_mat(x, "x", R, d, dt, dev),
          _vec(gamma, "gamma", d, dt, dev), _vec(beta, "beta", d, dt, dev), eps,
          *_mat(out, "out", R, d, dt, dev), _stats(stats, R, dev, False), _stream(stream, dev))


def norm_backward(plan: NormPlan, dout, x, gamma, stats, dx=None, dgamma=None, dbeta=None,
                  stream=None) -> None:
    if stream is None and plan._plain is not None and _taken(_short.norm_backward(
            plan._plain, dout, x, gamma, stats, dx, dgamma, dbeta, _current_stream(plan.device))):
        return
    R, d, dev, dt = _rows(dout, "dout"), plan.dim, plan.device, plan.dtype
    _call("route_norm_backward", plan, R, *_mat(dout, "dout", R, d, dt, dev),
          *_mat(x, "x", R, d, dt, dev), _vec(gamma, "gamma", d, dt, dev),
          _stats(stats, R, dev, True), *_opt_mat(dx, "dx", R, d, dt, dev),
          _vec(dgamma, "dgamma", d, dt, dev), _vec(dbeta, "dbeta", d, dt, dev),
          _stream(stream, dev))


def linear_forward(plan: LinearPlan, x, W, out, bias=None, residual=None, saved=None,
                   stream=None) -> None:
    if stream is None and plan._plain is not None and _taken(_short.linear_forward(
            plan._plain, x, W, out, bias, residual, saved, _current_stream(plan.device))):
        return
    R, k, n, dev, dt = _rows(x, "x"), plan.k, plan.n, plan.device, plan.dtype
    _call("route_linear_forward", plan, R, *_mat(x, "x", R, k, dt, dev),
          *_mat(W, "W", k, n, dt, dev), _vec(bias, "bias", n, dt, dev),
          *_opt_mat(residual, "residual", R, n, plan.out_dtype, dev),
          *_mat(out, "out", R, n, plan.out_dtype, dev), _saved(plan, saved, R),
          _stream(stream, dev))


def linear_backward(plan: LinearPlan, dout, x, W, saved=None, dx=None, dW=None, dbias=None,
                    stream=None) -> None:
    """`saved`: what the forward call kept (plans with an activation).  x may
    be None without dW, W without dx."""
    if stream is None and plan._plain is not None and _taken(_short.linear_backward(
            plan._plain, dout, x, W, saved, dx, dW, dbias, _current_stream(plan.device))):
        return
    R, k, n, dev, dt = _rows(dout, "dout"), plan.k, plan.n, plan.device, plan.dtype
    _call("route_linear_backward", plan, R, *_mat(dout, "dout", R, n, dt, dev),
          *_opt_mat(x, "x", R, k, dt, dev), *_opt_mat(W, "W", k, n, dt, dev),
          _saved(plan, saved, R), *_opt_mat(dx, "dx", R, k, dt, dev),
          *_opt_mat(dW, "dW", k, n, dt, dev), _vec(dbias, "dbias", n, dt, dev),
          _stream(stream, dev))


def gated_forward(plan: GatedPlan, x, W_gate, W_up, W_down, out, residual=None, saved=None,
                  stream=None) -> None:
    if stream is None and plan._plain is not None and _taken(_short.gated_forward(
            plan._plain, x, W_gate, W_up, W_down, out, residual, saved,
            _current_stream(plan.device))):
        return
    R, k, f, n, dev, dt = _rows(x, "x"), plan.k, plan.f, plan.n, plan.device, plan.dtype
    _call("route_gated_forward", plan, R, *_mat(x, "x", R, k, dt, dev),
          *_mat(W_gate, "W_gate", k, f, dt, dev), *_mat(W_up, "W_up", k, f, dt, dev),
          *_mat(W_down, "W_down", f, n, dt, dev), *_opt_mat(residual, "residual", R, n, dt, dev),
          *_mat(out, "out", R, n, dt, dev), _saved(plan, saved, R), _stream(stream, dev))


def gated_backward(plan: GatedPlan, dout, x, W_gate, W_up, W_down, saved, dx=None, dW_gate=None,
                   dW_up=None, dW_down=None, stream=None) -> None:
    if stream is None and plan._plain is not None and _taken(_short.gated_backward(
            plan._plain, dout, x, W_gate, W_up, W_down, saved, dx, dW_gate, dW_up,
            dW_down, _current_stream(plan.device))):
        return
    R, k, f, n, dev, dt = _rows(dout, "dout"), plan.k, plan.f, plan.n, plan.device, plan.dtype
    _call("route_gated_backward", plan, R, *_mat(dout, "dout", R, n, dt, dev),
          *_mat(x, "x", R, k, dt, dev), *_mat(W_gate, "W_gate", k, f, dt, dev),
          *_mat(W_up, "W_up", k, f, dt, dev), *_mat(W_down, "W_down", f, n, dt, dev),
          _saved(plan, saved, R), *_opt_mat(dx, "dx", R, k, dt, dev),
          *_opt_mat(dW_gate, "dW_gate", k, f, dt, dev), *_opt_mat(dW_up, "dW_up", k, f, dt, dev),
          *_opt_mat(dW_down, "dW_down", f, n, dt, dev), _stream(stream, dev))
