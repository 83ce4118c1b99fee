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
_torch = None
_types = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes = [_vp, _vp]
        f.restype = _int
        _fns[name] = f
    return f


def _setup():
    global _torch
    import torch
    _types.update({torch.float16: 2, torch.bfloat16: 3, torch.float32: 4})
    _torch = torch


def _bad(why):
    raise RingarError(INVALID_ARGUMENT, why)


def _type(t):
    if _torch is None:
        _setup()
    code = _types.get(t.dtype)
    if code is None:
        _bad(f"unsupported dtype {t.dtype}: float16, bfloat16 or float32")
    return code


def _rows(t, what, like=None):
    """(rows, columns, row stride) of a tensor whose last dimension is contiguous."""
    if not t.is_cuda:
        _bad(f"{what} must be a CUDA tensor")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        _bad(f"{what} must have the dtype and device of the other operands")
    shape, stride = t.shape, t.stride()
    n = len(shape)
    if n == 0:
        _bad(f"{what} needs at least one dimension")
    cols = shape[-1]
    if cols > 1 and stride[-1] != 1:
        _bad(f"{what}: the last dimension must be contiguous")
    if n == 2:
        rows = shape[0]
        return rows, cols, stride[0] if rows > 1 else cols
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
    if t.dtype != dtype or t.device != device or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        _bad(f"{what} must be a contiguous vector of {n} values of {dtype} on the operands' GPU")
    return t.data_ptr()


class _On:
    """The stream a call runs on; tensors made inside belong to it, and
    ``uses`` keeps the caller's tensors alive until its work is done where it
    is not their own."""

    def __init__(self, x, stream):
        self.device = x.device.index
        self.other = None
        if stream is not None and stream.cuda_stream != _torch._C._cuda_getCurrentRawStream(self.device):
            self.other = _torch.cuda.stream(stream)
            self.stream = stream
        elif self.device != _torch.cuda.current_device():
            self.other = _torch.cuda.device(self.device)
            self.stream = None

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()
        return self

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)

    def call(self, name, args, *tensors):
        code = _fn(name)(ctypes.byref(args), _torch._C._cuda_getCurrentRawStream(self.device))
        if code != SUCCESS:
            raise RingarError(code, f"{name} ({ringar_last_error()})")
        if self.other is not None and self.stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _out(out, like, shape, what):
    if out is None:
        return _torch.empty(shape, dtype=like.dtype, device=like.device)
    if tuple(out.shape) != tuple(shape):
        _bad(f"{what} must have shape {tuple(shape)}")
    return out


def layer_norm(x, weight=None, bias=None, eps=1e-5, *, stats=False, out=None, stream=None):
    """``(x - mean) * rstd * weight + bias`` over the last dimension.

    ``weight`` and ``bias``: vectors of x's dtype or both float32.  ``stats``:
    return ``(y, mean, rstd)``, the float32 row statistics that
    ``layer_norm_backward`` takes.  ``out``: where y goes (it may be x)."""
    code = _type(x)
    rows, cols, ldx = _rows(x, "x")
    p = weight if weight is not None else bias
    pdtype = x.dtype if p is None else p.dtype
    w = _vector(weight, cols, "weight", pdtype, x.device)
    b = _vector(bias, cols, "bias", pdtype, x.device)
    with _On(x, stream) as on:
        y = _out(out, x, x.shape, "out")
        ldy = _rows(y, "out", x)[2]
        mean = rstd = None
        if stats:
            mean = _torch.empty(x.shape[:-1], dtype=_torch.float32, device=x.device)
            rstd = _torch.empty_like(mean)
        on.call("ringar_layer_norm",
                ringar_layer_norm_t(code, code if p is None else _type(p), rows, cols, x.data_ptr(), ldx, w, b, eps,
                                    y.data_ptr(), ldy, _ptr(mean), _ptr(rstd)), x, weight, bias, out)
    return (y, mean, rstd) if stats else y


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, dx=True, dweight=True, dbias=True, stream=None):
    """``(dx, dweight, dbias)`` of ``layer_norm``; one whose flag is False is
    not computed and None.  The parameter gradients have the weight's dtype
    (x's without a weight)."""
    code = _type(x)
    rows, cols, ldx = _rows(x, "x")
    r2, c2, lddy = _rows(dy, "dy", x)
    if (r2, c2) != (rows, cols):
        _bad("dy must have x's shape")
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != _torch.float32 or t.numel() != rows or not t.is_contiguous() or t.device != x.device:
            _bad(f"{what} must be {rows} contiguous float32 values on x's GPU")
    pdtype = x.dtype if weight is None else weight.dtype
    w = _vector(weight, cols, "weight", pdtype, x.device)
    with _On(x, stream) as on:
        gx = _torch.empty(x.shape, dtype=x.dtype, device=x.device) if dx else None
        gw = _torch.empty(cols, dtype=pdtype, device=x.device) if dweight else None
        gb = _torch.empty(cols, dtype=pdtype, device=x.device) if dbias else None
        on.call("ringar_layer_norm_backward",
                ringar_layer_norm_backward_t(code, code if weight is None else _type(weight), rows, cols,
                                             dy.data_ptr(), lddy, x.data_ptr(), ldx, mean.data_ptr(),
                                             rstd.data_ptr(), w, _ptr(gx), cols, _ptr(gw), _ptr(gb)),
                dy, x, mean, rstd, weight)
    return gx, gw, gb


def _forward(name, gated, x, weight, bias, act, residual, save_pre, out, stream):
    code = _type(x)
    if act not in ACTS:
        _bad(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
    rows, k, ldx = _rows(x, "x")
    if weight.dim() != 2:
        _bad("weight must have two dimensions")
    wide, k2, ldw = _rows(weight, "weight", x)
    if k2 != k or (gated and wide % 2):
        _bad("weight must be out_features x in_features" if not gated else "weight must be 2 out_features x in_features")
    n = wide // 2 if gated else wide
    b = _vector(bias, wide, "bias", x.dtype, x.device)
    ldr = 0
    if residual is not None:
        rr, rc, ldr = _rows(residual, "residual", x)
        if (rr, rc) != (rows, n):
            _bad("residual must have the output's shape")
    lead = x.shape[:-1]
    with _On(x, stream) as on:
        y = _out(out, x, (*lead, n), "out")
        ldy = _rows(y, "out", x)[2]
        pre = _torch.empty((*lead, wide), dtype=x.dtype, device=x.device) if save_pre else None
        on.call(name, ringar_linear_t(code, ACTS[act], rows, k, n, x.data_ptr(), ldx, weight.data_ptr(), ldw, b,
                                      _ptr(residual), ldr, y.data_ptr(), ldy, _ptr(pre), wide),
                x, weight, bias, residual, out)
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
    code = _type(dy)
    if act not in ACTS:
        _bad(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
    rows, n, lddy = _rows(dy, "dy")
    wide = 2 * n if gated else n
    px = pw = pp = None
    ldx = ldw = ldp = k = 0
    if x is not None:
        rx, k, ldx = _rows(x, "x", dy)
        px = x.data_ptr()
        if rx != rows:
            _bad("x and dy must have the same rows")
    elif dweight:
        _bad("the weight's gradient needs x")
    if weight is not None:
        rw, kw, ldw = _rows(weight, "weight", dy)
        pw = weight.data_ptr()
        if rw != wide or weight.dim() != 2 or (x is not None and kw != k):
            _bad("weight does not fit dy and x")
        k = kw
    elif dx:
        _bad("x's gradient needs the weight")
    if pre is not None:
        rp, cp, ldp = _rows(pre, "pre", dy)
        pp = pre.data_ptr()
        if (rp, cp) != (rows, wide):
            _bad(f"pre must have {wide} columns and dy's rows")
    elif gated or act != "none":
        _bad("pre, kept by the forward pass, is needed")
    with _On(dy, stream) as on:
        kw = dict(dtype=dy.dtype, device=dy.device)
        gx = _torch.empty((*dy.shape[:-1], k), **kw) if dx else None
        gw = _torch.empty((wide, k), **kw) if dweight else None
        gb = _torch.empty(wide, **kw) if dbias else None
        on.call(name, ringar_linear_backward_t(code, ACTS[act], rows, k, n, dy.data_ptr(), lddy, pp, ldp, px, ldx,
                                               pw, ldw, _ptr(gx), k, _ptr(gw), k, _ptr(gb)), dy, x, weight, pre)
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
