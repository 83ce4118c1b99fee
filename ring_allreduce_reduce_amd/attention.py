"""Cross attention on torch tensors: queries of a decoder to the states of an
encoder, whose length is another (the C calls and their formulas are in
include/ringar.h).

Tensors are CUDA tensors of one GPU and one dtype (fp16, bf16 or fp32), of
shape (batch, rows, heads, head_dim) at any strides whose rows start at
16-byte boundaries: what a projection leaves, one projection's halves, or a
``transpose(1, 2)`` of heads before rows.  As the block operators, a call
enqueues on ``stream`` (default: the current one), returns new tensors, and is
not recorded by autograd.
"""
from __future__ import annotations

from . import block
from .block import _float, _i64, _int, _On, _struct, _vp

_three = _i64 * 3

ringar_cross_attention_t = _struct(
    "ringar_cross_attention_t", ("dtype", _int), ("batch", _i64), ("queries", _i64), ("keys", _i64), ("heads", _i64),
    ("kv_heads", _i64), ("head_dim", _i64), ("q", _vp), ("q_strides", _three), ("k", _vp), ("k_strides", _three), ("v", _vp),
    ("v_strides", _three), ("key_lengths", _vp), ("scale", _float), ("y", _vp), ("y_strides", _three), ("lse", _vp))
ringar_cross_attention_backward_t = _struct(
    "ringar_cross_attention_backward_t", ("dtype", _int), ("batch", _i64), ("queries", _i64), ("keys", _i64), ("heads", _i64),
    ("kv_heads", _i64), ("head_dim", _i64), ("dy", _vp), ("dy_strides", _three), ("q", _vp), ("q_strides", _three), ("k", _vp),
    ("k_strides", _three), ("v", _vp), ("v_strides", _three), ("y", _vp), ("y_strides", _three), ("lse", _vp),
    ("key_lengths", _vp), ("scale", _float), ("dq", _vp), ("dk", _vp), ("dv", _vp))


def cross_attention(q, k, v, *, key_lengths=None, scale=None, stats=False, out=None, stream=None):
    """``softmax(scale * q @ k^T) @ v`` for every sequence and head, shaped like q.

    q: (batch, queries, heads, head_dim); k and v: (batch, keys, kv_heads,
    head_dim), kv_heads dividing heads (neighbouring query heads share a key
    head).  head_dim: a multiple of 8 (float32: 4) up to 128.  ``key_lengths``:
    int32, the keys of each sequence (default: all; a value outside 0 .. keys
    counts as the nearer end); keys past them are not looked at, whatever they
    hold.  A row without keys is zero.  ``scale``: 1 / sqrt(head_dim) by default.
    ``stats``: return ``(y, lse)``, the float32 log-sums of shape (batch, heads,
    queries) that ``cross_attention_backward`` takes.  ``out``: where y goes."""
    ext = block._ext or block._load()
    if stream is None:
        return ext.cross_attention(q, k, v, key_lengths, scale, stats, out)
    with _On(stream, q, k, v, key_lengths, out):
        return ext.cross_attention(q, k, v, key_lengths, scale, stats, out)


def cross_attention_backward(dy, q, k, v, y, lse, *, key_lengths=None, scale=None, dq=True, dk=True, dv=True, stream=None):
    """``(dq, dk, dv)`` of ``cross_attention``; one whose flag is False is None.
    (dk and dv are computed together: one of them alone takes as long as both.)
    ``y``, ``lse``: the forward pass's; ``key_lengths`` and ``scale`` as there.
    Keys past a sequence's length get zeros."""
    ext = block._ext or block._load()
    if stream is None:
        return ext.cross_attention_backward(dy, q, k, v, y, lse, key_lengths, scale, dq, dk, dv)
    with _On(stream, dy, q, k, v, y, lse, key_lengths):
        return ext.cross_attention_backward(dy, q, k, v, y, lse, key_lengths, scale, dq, dk, dv)
