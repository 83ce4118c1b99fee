"""Block operators on torch tensors: layer norm, the linear product with bias,
activation and residual, and the gated feed-forward, each with its backward
pass (the C calls and their formulas are in include/ringar.h).

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
