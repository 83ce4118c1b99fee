"""Block operators on torch tensors: layer norm, the root-mean-square norm
joined to the residual stream, the linear product with bias, activation and
residual, the gated feed-forward, and dropout, each with its backward pass (the
C calls and their formulas are in include/ringar.h; cross attention is in
attention.py).

They are what a tensor-parallel transformer block computes between two
AllReduces.  Tensors are CUDA tensors of one GPU whose last dimension is
contiguous; the dimensions before it are rows (a view that does not collapse
to one row stride is refused, never copied).  A call enqueues on ``stream`` (a
torch stream; default: the current one) and returns the output tensors; it is
not recorded by autograd, whatever its inputs require: gradients come from the
``_backward`` calls.  A tensor given as ``out`` counts as changed in place.
"""
from __future__ import annotations

import ctypes
import os

from . import HERE, INTERNAL, INVALID_ARGUMENT, RingarError, load

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
ringar_rms_norm_t = _struct(
    "ringar_rms_norm_t", ("dtype", _int), ("param_dtype", _int), ("out", _int), ("rows", _i64), ("cols", _i64), ("x", _vp),
    ("ldx", _i64), ("residual", _vp), ("ldr", _i64), ("weight", _vp), ("eps", _float), ("sum", _vp), ("lds", _i64),
    ("y", _vp), ("ldy", _i64), ("scale", _vp), ("rstd", _vp))
ringar_rms_norm_backward_t = _struct(
    "ringar_rms_norm_backward_t", ("dtype", _int), ("param_dtype", _int), ("rows", _i64), ("cols", _i64), ("dy", _vp),
    ("lddy", _i64), ("x", _vp), ("ldx", _i64), ("rstd", _vp), ("weight", _vp), ("dsum", _vp), ("ldds", _i64),
    ("dx", _vp), ("lddx", _i64), ("dweight", _vp))
ringar_dropout_t = _struct(
    "ringar_dropout_t", ("dtype", _int), ("rows", _i64), ("cols", _i64), ("x", _vp), ("ldx", _i64), ("residual", _vp),
    ("ldr", _i64), ("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("more_offset", _vp),
    ("first_row", _i64), ("first_col", _i64), ("y", _vp), ("ldy", _i64))

_fns = {}
_ext = None


def _fn(name):
    """The C entry ``name`` of the library."""
    f = _fns.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes = [_vp, _vp]
        f.restype = _int
        _fns[name] = f
    return f


def _load():
    """The extension that checks tensors, makes the outputs and calls the
    library (built by ``__graft_entry__.build()``; there is no fallback)."""
    global _ext
    import torch  # noqa: F401  (its libraries first)
    load()
    path = os.path.join(HERE, "_block_ext.so")
    if not os.path.exists(path):
        raise RingarError(INTERNAL, f"{path} is missing; build it with __graft_entry__.build()")
    from . import _block_ext
    _ext = _block_ext
    return _ext


def _act(name):
    code = ACTS.get(name) if isinstance(name, str) else None
    if code is None:
        raise RingarError(INVALID_ARGUMENT, f"unknown activation {name!r}: one of {', '.join(ACTS)}")
    return code


class _On:
    """Runs a call on a stream: outputs are made there, and the caller's
    tensors are kept until its work is done."""

    def __init__(self, stream, *tensors):
        import torch
        for t in tensors:
            if t is not None and not isinstance(t, torch.Tensor):
                raise RingarError(INVALID_ARGUMENT, f"a tensor is needed, not {type(t).__name__}")
            if t is not None and t.is_cuda and t.get_device() != stream.device_index:
                raise RingarError(INVALID_ARGUMENT, "the stream belongs to another GPU than the operands")
        self.stream, self.tensors, self.on = stream, tensors, torch.cuda.stream(stream)

    def __enter__(self):
        self.on.__enter__()

    def __exit__(self, *exc):
        if exc[0] is None:
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)
        self.on.__exit__(*exc)


def layer_norm(x, weight=None, bias=None, eps=1e-5, *, stats=False, out=None, stream=None):
    """``(x - mean) * rstd * weight + bias`` over the last dimension.

    ``weight`` and ``bias``: vectors of x's dtype or both float32.  ``stats``:
    return ``(y, mean, rstd)``, the float32 row statistics that
    ``layer_norm_backward`` takes.  ``out``: where y goes (it may be x)."""
    ext = _ext or _load()
    if stream is None:
        return ext.layer_norm(x, weight, bias, eps, stats, out)
    with _On(stream, x, weight, bias, out):
        return ext.layer_norm(x, weight, bias, eps, stats, out)


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, dx=True, dweight=True, dbias=True, stream=None):
    """``(dx, dweight, dbias)`` of ``layer_norm``; one whose flag is False is
    not computed and None.  The parameter gradients have the weight's dtype
    (x's without a weight)."""
    ext = _ext or _load()
    if stream is None:
        return ext.layer_norm_backward(dy, x, mean, rstd, weight, dx, dweight, dbias)
    with _On(stream, dy, x, mean, rstd, weight):
        return ext.layer_norm_backward(dy, x, mean, rstd, weight, dx, dweight, dbias)


def rms_norm(x, weight=None, eps=1e-6, *, residual=None, stats=False, out=None, sum_out=None, stream=None):
    """``s * rstd * weight`` over the last dimension, ``rstd = 1 / sqrt(mean(s^2)
    + eps)``, with ``s = x + residual`` rounded to x's dtype (x itself without a
    residual).

    Returns y, or with a residual or ``stats`` a tuple: y, s (with a residual),
    the float32 rstd (with ``stats``); s and rstd are what ``rms_norm_backward``
    takes.  ``weight``: of x's dtype or float32.  ``out`` and ``sum_out``: where
    y and s go (each may be x or the residual)."""
    ext = _ext or _load()
    if stream is None:
        return ext.rms_norm(x, weight, eps, residual, 0, stats, out, sum_out)
    with _On(stream, x, weight, residual, out, sum_out):
        return ext.rms_norm(x, weight, eps, residual, 0, stats, out, sum_out)


def rms_norm_fp8(x, weight=None, eps=1e-6, *, residual=None, group=None, stats=False, sum_out=None, stream=None):
    """``rms_norm`` with y in 8 bits: a tuple of q (float8_e4m3fn), the float32
    scale that q's values stand at, and s and rstd as there.

    ``group``: None for one scale a row (``scale`` of shape x.shape[:-1] +
    (1,)), or 128 for one for every 128 columns (x.shape[:-1] + (ceil(cols /
    128),)).  A scale is the largest magnitude of its values / 448."""
    ext = _ext or _load()
    if group is not None and (isinstance(group, bool) or group != 128):
        raise RingarError(INVALID_ARGUMENT, f"group must be None (a row) or 128 columns, not {group!r}")
    kind = 1 if group is None else 2
    if stream is None:
        return ext.rms_norm(x, weight, eps, residual, kind, stats, None, sum_out)
    with _On(stream, x, weight, residual, sum_out):
        return ext.rms_norm(x, weight, eps, residual, kind, stats, None, sum_out)


def rms_norm_backward(dy, x, rstd, weight=None, *, dsum=None, dx=True, dweight=True, stream=None):
    """``(dx, dweight)`` of ``rms_norm``; one whose flag is False is not computed
    and None.  ``x``: the forward pass's s.  ``dsum``: the gradient that reaches
    s on the residual stream's own way; it is added to dx, which is the gradient
    of x and of the residual alike.  ``dweight`` has the weight's dtype (x's
    without a weight)."""
    ext = _ext or _load()
    if stream is None:
        return ext.rms_norm_backward(dy, x, rstd, weight, dsum, dx, dweight)
    with _On(stream, dy, x, rstd, weight, dsum):
        return ext.rms_norm_backward(dy, x, rstd, weight, dsum, dx, dweight)


def dropout(x, p, seed, offset=0, *, residual=None, first_row=0, first_col=0, out=None, stream=None):
    """``where(keep, x / (1 - p), 0) + residual`` with a mask that is computed,
    never stored: from ``seed`` and ``offset`` (0 .. 2^64 - 1; another offset is
    another mask), a value's row and its column.

    ``offset`` may be an int64 tensor of one value on x's GPU: a captured call
    reads it at every replay.  ``first_row``, ``first_col`` (a multiple of 8):
    where x lies in a larger array, whose mask it then has.  p is rounded to 16
    bits.  ``out``: where y goes (it may be x or the residual)."""
    ext = _ext or _load()
    if stream is None:
        return ext.dropout(x, p, seed, offset, residual, first_row, first_col, out)
    with _On(stream, x, residual, out, offset if not isinstance(offset, int) else None):
        return ext.dropout(x, p, seed, offset, residual, first_row, first_col, out)


def dropout_backward(dy, p, seed, offset=0, *, first_row=0, first_col=0, out=None, stream=None):
    """The gradient of ``dropout``'s x: the same mask and scale on dy.  (The
    residual's gradient is dy itself.)"""
    return dropout(dy, p, seed, offset, first_row=first_row, first_col=first_col, out=out, stream=stream)


def linear(x, weight, bias=None, *, act="none", residual=None, save_pre=False, out=None, stream=None):
    """``act(x @ weight.T + bias) + residual`` with ``weight`` of shape
    (out_features, in_features).  ``save_pre``: return ``(y, pre)``, the
    pre-activation that ``linear_backward`` takes.  ``out``: where y goes (it
    may be the residual)."""
    ext, act = _ext or _load(), _act(act)
    if stream is None:
        return ext.forward(x, weight, bias, act, residual, save_pre, out, False)
    with _On(stream, x, weight, bias, residual, out):
        return ext.forward(x, weight, bias, act, residual, save_pre, out, False)


def gated_ffn(x, weight, bias=None, *, act="silu", save_pre=False, out=None, stream=None):
    """``act(x @ Wg.T + bg) * (x @ Wu.T + bu)`` with ``weight`` the gate's
    out_features rows and then the up projection's, ``bias`` likewise.
    ``save_pre``: return ``(h, pre)``, pre = both projections side by side."""
    ext, act = _ext or _load(), _act(act)
    if stream is None:
        return ext.forward(x, weight, bias, act, None, save_pre, out, True)
    with _On(stream, x, weight, bias, out):
        return ext.forward(x, weight, bias, act, None, save_pre, out, True)


def linear_backward(dy, x, weight, pre=None, *, act="none", dx=True, dweight=True, dbias=True, stream=None):
    """``(dx, dweight, dbias)`` of ``linear``; one whose flag is False is not
    computed and None (x is needed for dweight, weight for dx).  ``pre``: the
    forward pass's pre-activation, needed with an activation.  The residual's
    gradient is dy itself."""
    ext, act = _ext or _load(), _act(act)
    if stream is None:
        return ext.backward(dy, x, weight, pre, act, dx, dweight, dbias, False)
    with _On(stream, dy, x, weight, pre):
        return ext.backward(dy, x, weight, pre, act, dx, dweight, dbias, False)


def gated_ffn_backward(dy, x, weight, pre, *, act="silu", dx=True, dweight=True, dbias=True, stream=None):
    """``(dx, dweight, dbias)`` of ``gated_ffn``, as ``linear_backward``."""
    ext, act = _ext or _load(), _act(act)
    if stream is None:
        return ext.backward(dy, x, weight, pre, act, dx, dweight, dbias, True)
    with _On(stream, dy, x, weight, pre):
        return ext.backward(dy, x, weight, pre, act, dx, dweight, dbias, True)
