"""Block operators on torch tensors: layer norm, the linear product with bias,
activation and residual, and the gated feed-forward, each with its backward
pass (the C calls and their formulas are in include/ringar.h).

They are what a tensor-parallel transformer block computes between two
AllReduces.  Tensors are CUDA tensors of one GPU whose last dimension is
contiguous; the dimensions before it are rows (a view that does not collapse
to one row stride is refused, never copied).  A call enqueues on ``stream`` (a
torch stream; default: the current one) and returns the output tensors; it is
not recorded by autograd: gradients come from the ``_backward`` calls.
"""
from __future__ import annotations

import ctypes

from . import INVALID_ARGUMENT, SUCCESS, RingarError, load, ringar_last_error

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "sigmoid": 5}

_vp, _i64, _int, _float = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float


def _struct(name, *fields):
    return type(name, (ctypes.Structure,), {"_fields_": list(fields)})


ringar_layer_norm_t = _struct(
    "ringar_layer_norm_t", ("dtype", _int), ("param_dtype", _int), ("rows", _i64), ("cols", _i64), ("x", _vp),
    ("ldx", _i64), ("weight", _vp), ("bias", _vp), ("eps", _float), ("y", _vp), ("ldy", _i64), ("mean", _vp),
    ("rstd", _vp))
ringar_layer_norm_backward_t = _struct(
    "ringar_layer_norm_backward_t", ("dtype", _int), ("param_dtype", _int), ("rows", _i64), ("cols", _i64),
    ("dy", _vp), ("lddy", _i64), ("x", _vp), ("ldx", _i64), ("mean", _vp), ("rstd", _vp), ("weight", _vp),
    ("dx", _vp), ("lddx", _i64), ("dweight", _vp), ("dbias", _vp))
ringar_linear_t = _struct(
    "ringar_linear_t", ("dtype", _int), ("act", _int), ("rows", _i64), ("in_features", _i64),
    ("out_features", _i64), ("x", _vp), ("ldx", _i64), ("weight", _vp), ("ldw", _i64), ("bias", _vp),
    ("residual", _vp), ("ldr", _i64), ("y", _vp), ("ldy", _i64), ("pre", _vp), ("ldp", _i64))
ringar_linear_backward_t = _struct(
    "ringar_linear_backward_t", ("dtype", _int), ("act", _int), ("rows", _i64), ("in_features", _i64),
    ("out_features", _i64), ("dy", _vp), ("lddy", _i64), ("pre", _vp), ("ldp", _i64), ("x", _vp), ("ldx", _i64),
    ("weight", _vp), ("ldw", _i64), ("dx", _vp), ("lddx", _i64), ("dweight", _vp), ("lddw", _i64), ("dbias", _vp))

_fns = {}
_types = {}
_torch = _device_now = _stream_now = None


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes = [_vp, _vp]
        f.restype = _int
        _fns[name] = f
    return f


def _setup():
    global _torch, _device_now, _stream_now
    import torch
    torch.cuda.init()
    _types.update({torch.float16: 2, torch.bfloat16: 3, torch.float32: 4})
    _device_now, _stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _torch = torch


def _bad(why):
    raise RingarError(INVALID_ARGUMENT, why)


def _begin(x):
    """(dtype, its code, device index) of the operand that the others go by."""
    device = x.get_device()
    if device < 0:
        _bad("the operands must be CUDA tensors")
    if _torch is None:
        _setup()
    dtype = x.dtype
    code = _types.get(dtype)
    if code is None:
        _bad(f"unsupported dtype {dtype}: float16, bfloat16 or float32")
    return dtype, code, device


def _rows(t, what, dtype, device):
    """(rows, columns, row stride) of a tensor whose last dimension is contiguous."""
    if t.dtype is not dtype or t.get_device() != device:
        _bad(f"{what} must have the dtype and device of the other operands")
    shape, stride = t.shape, t.stride()
    n = len(shape)
    if n == 2:
        rows, cols = shape
        if stride[1] != 1 and cols > 1:
            _bad(f"{what}: the last dimension must be contiguous")
        return rows, cols, stride[0] if rows > 1 else cols
    if n == 0:
        _bad(f"{what} needs at least one dimension")
    cols = shape[-1]
    if cols > 1 and stride[-1] != 1:
        _bad(f"{what}: the last dimension must be contiguous")
    rows, ld = 1, None
    for size, step in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if size == 0:
            return 0, cols, cols
        if size == 1:
            continue
        if ld is None:
            ld = step
        elif step != rows * ld:
            _bad(f"{what}: the rows must lie at one stride (make the tensor contiguous first)")
        rows *= size
    return rows, cols, cols if ld is None else ld


def _vector(t, n, what, dtype, device):
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or t.shape != (n,) or not t.is_contiguous():
        _bad(f"{what} must be a contiguous vector of {n} values of {dtype} on the operands' GPU")
    return t.data_ptr()


def _call(name, args, device):
    code = _fn(name)(ctypes.byref(args), _stream_now(device))
    if code != SUCCESS:
        raise RingarError(code, f"{name} ({ringar_last_error()})")


class _Elsewhere:
    """Runs a call on another stream or GPU than the current one: outputs are
    made there, and the caller's tensors are kept until its work is done."""

    def __init__(self, device, stream, *tensors):
        self.device, self.stream, self.tensors = _torch.cuda.device(device), stream, tensors
        if stream is not None and stream.device_index != device:
            _bad("the stream belongs to another GPU than the operands")
        self.on = _torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        self.on.__enter__()

    def __exit__(self, *exc):
        if exc[0] is None and self.stream is not None:
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)
        self.on.__exit__(*exc)
        self.device.__exit__(*exc)


def _ptr(t):
    return None if t is None else t.data_ptr()


def layer_norm(x, weight=None, bias=None, eps=1e-5, *, stats=False, out=None, stream=None):
    """``(x - mean) * rstd * weight + bias`` over the last dimension.

    ``weight`` and ``bias``: vectors of x's dtype or both float32.  ``stats``:
    return ``(y, mean, rstd)``, the float32 row statistics that
    ``layer_norm_backward`` takes.  ``out``: where y goes (it may be x)."""
    dtype, code, device = _begin(x)
    if stream is not None or device != _device_now():
        with _Elsewhere(device, stream, x, weight, bias, out):
            return layer_norm(x, weight, bias, eps, stats=stats, out=out)
    rows, cols, ldx = _rows(x, "x", dtype, device)
    p = weight if weight is not None else bias
    pdtype = dtype if p is None else p.dtype
    w = _vector(weight, cols, "weight", pdtype, device)
    b = _vector(bias, cols, "bias", pdtype, device)
    if out is None:
        y, ldy = x.new_empty(x.shape), cols
    else:
        y, ldy = out, _rows(out, "out", dtype, device)[2]
        if out.shape != x.shape:
            _bad("out must have x's shape")
    mean = rstd = None
    if stats:
        mean = _torch.empty(x.shape[:-1], dtype=_torch.float32, device=x.device)
        rstd = _torch.empty_like(mean)
    _call("ringar_layer_norm",
          ringar_layer_norm_t(code, _types.get(pdtype, -1), rows, cols, x.data_ptr(), ldx, w, b, eps, y.data_ptr(), ldy,
                              _ptr(mean), _ptr(rstd)), device)
    return (y, mean, rstd) if stats else y


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, dx=True, dweight=True, dbias=True, stream=None):
    """``(dx, dweight, dbias)`` of ``layer_norm``; one whose flag is False is
    not computed and None.  The parameter gradients have the weight's dtype
    (x's without a weight)."""
    dtype, code, device = _begin(x)
    if stream is not None or device != _device_now():
        with _Elsewhere(device, stream, dy, x, mean, rstd, weight):
            return layer_norm_backward(dy, x, mean, rstd, weight, dx=dx, dweight=dweight, dbias=dbias)
    rows, cols, ldx = _rows(x, "x", dtype, device)
    r2, c2, lddy = _rows(dy, "dy", dtype, device)
    if r2 != rows or c2 != cols:
        _bad("dy must have x's shape")
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype is not _torch.float32 or t.numel() != rows or not t.is_contiguous() or t.get_device() != device:
            _bad(f"{what} must be {rows} contiguous float32 values on x's GPU")
    pdtype = dtype if weight is None else weight.dtype
    w = _vector(weight, cols, "weight", pdtype, device)
    gx = x.new_empty(x.shape) if dx else None
    gw = x.new_empty(cols, dtype=pdtype) if dweight else None
    gb = x.new_empty(cols, dtype=pdtype) if dbias else None
    _call("ringar_layer_norm_backward",
          ringar_layer_norm_backward_t(code, _types.get(pdtype, -1), rows, cols, dy.data_ptr(), lddy, x.data_ptr(), ldx,
                                       mean.data_ptr(), rstd.data_ptr(), w, _ptr(gx), cols, _ptr(gw), _ptr(gb)), device)
    return gx, gw, gb


def _forward(name, gated, x, weight, bias, act, residual, save_pre, out, stream):
    dtype, code, device = _begin(x)
    if stream is not None or device != _device_now():
        with _Elsewhere(device, stream, x, weight, bias, residual, out):
            return _forward(name, gated, x, weight, bias, act, residual, save_pre, out, None)
    a = ACTS.get(act)
    if a is None:
        _bad(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
    rows, k, ldx = _rows(x, "x", dtype, device)
    wide, k2, ldw = _rows(weight, "weight", dtype, device)
    if k2 != k or weight.dim() != 2 or (gated and wide % 2):
        _bad("weight must be out_features x in_features" if not gated else "weight must be 2 out_features x in_features")
    n = wide // 2 if gated else wide
    b = _vector(bias, wide, "bias", dtype, device)
    r, ldr = None, 0
    if residual is not None:
        rr, rc, ldr = _rows(residual, "residual", dtype, device)
        if rr != rows or rc != n:
            _bad("residual must have the output's shape")
        r = residual.data_ptr()
    lead = x.shape[:-1]
    if out is None:
        y, ldy = x.new_empty((*lead, n)), n
    else:
        y, ldy = out, _rows(out, "out", dtype, device)[2]
        if out.shape != (*lead, n):
            _bad(f"out must have shape {(*lead, n)}")
    pre = x.new_empty((*lead, wide)) if save_pre else None
    _call(name, ringar_linear_t(code, a, rows, k, n, x.data_ptr(), ldx, weight.data_ptr(), ldw, b, r, ldr, y.data_ptr(),
                                ldy, _ptr(pre), wide), device)
    return (y, pre) if save_pre else y


def linear(x, weight, bias=None, *, act="none", residual=None, save_pre=False, out=None, stream=None):
    """``act(x @ weight.T + bias) + residual`` with ``weight`` of shape
    (out_features, in_features).  ``save_pre``: return ``(y, pre)``, the
    pre-activation that ``linear_backward`` takes.  ``out``: where y goes (it
    may be the residual)."""
    return _forward("ringar_linear", False, x, weight, bias, act, residual, save_pre, out, stream)


def gated_ffn(x, weight, bias=None, *, act="silu", save_pre=False, out=None, stream=None):
    """``act(x @ Wg.T + bg) * (x @ Wu.T + bu)`` with ``weight`` the gate's
    out_features rows and then the up projection's, ``bias`` likewise.
    ``save_pre``: return ``(h, pre)``, pre = both projections side by side."""
    return _forward("ringar_gated_ffn", True, x, weight, bias, act, None, save_pre, out, stream)


def _backward(name, gated, dy, x, weight, pre, act, dx, dweight, dbias, stream):
    dtype, code, device = _begin(dy)
    if stream is not None or device != _device_now():
        with _Elsewhere(device, stream, dy, x, weight, pre):
            return _backward(name, gated, dy, x, weight, pre, act, dx, dweight, dbias, None)
    a = ACTS.get(act)
    if a is None:
        _bad(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
    rows, n, lddy = _rows(dy, "dy", dtype, device)
    wide = 2 * n if gated else n
    px = pw = pp = None
    ldx = ldw = ldp = k = 0
    if x is not None:
        rx, k, ldx = _rows(x, "x", dtype, device)
        px = x.data_ptr()
        if rx != rows:
            _bad("x and dy must have the same rows")
    elif dweight:
        _bad("the weight's gradient needs x")
    if weight is not None:
        rw, kw, ldw = _rows(weight, "weight", dtype, device)
        pw = weight.data_ptr()
        if rw != wide or weight.dim() != 2 or (x is not None and kw != k):
            _bad("weight does not fit dy and x")
        k = kw
    elif dx:
        _bad("x's gradient needs the weight")
    if pre is not None:
        rp, cp, ldp = _rows(pre, "pre", dtype, device)
        pp = pre.data_ptr()
        if rp != rows or cp != wide:
            _bad(f"pre must have {wide} columns and dy's rows")
    elif gated or a:
        _bad("pre, kept by the forward pass, is needed")
    gx = dy.new_empty((*dy.shape[:-1], k)) if dx else None
    gw = dy.new_empty((wide, k)) if dweight else None
    gb = dy.new_empty(wide) if dbias else None
    _call(name, ringar_linear_backward_t(code, a, rows, k, n, dy.data_ptr(), lddy, pp, ldp, px, ldx, pw, ldw, _ptr(gx), k,
                                         _ptr(gw), k, _ptr(gb)), device)
    return gx, gw, gb


def linear_backward(dy, x, weight, pre=None, *, act="none", dx=True, dweight=True, dbias=True, stream=None):
    """``(dx, dweight, dbias)`` of ``linear``; one whose flag is False is not
    computed and None (x is needed for dweight, weight for dx).  ``pre``: the
    forward pass's pre-activation, needed with an activation.  The residual's
    gradient is dy itself."""
    return _backward("ringar_linear_backward", False, dy, x, weight, pre, act, dx, dweight, dbias, stream)


def gated_ffn_backward(dy, x, weight, pre, *, act="silu", dx=True, dweight=True, dbias=True, stream=None):
    """``(dx, dweight, dbias)`` of ``gated_ffn``, as ``linear_backward``."""
    return _backward("ringar_gated_ffn_backward", True, dy, x, weight, pre, act, dx, dweight, dbias, stream)
