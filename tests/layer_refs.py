"""Plain fp64 forms of the root-mean-square norm, dropout and cross attention,
each with a bound on what a correct kernel may differ by (the arithmetic that
the bounds count is block_refs.py's: fp32 sums, one rounding of an output)."""
import math

import numpy as np
import torch

from block_refs import TINY, U32, UNIT, _depth, rounded

LARGEST = 448.0


# ------------------------------------------------------------------ rms norm
def rms_forward(s, w, eps):
    """y, rstd of the norm of ``s`` and their bounds, before y's rounding."""
    s = s.double().cpu().reshape(-1, s.shape[-1])
    cols = s.shape[1]
    w = torch.ones(cols, dtype=torch.float64) if w is None else w.double().cpu()
    mean = (s * s).mean(1)
    rstd = 1 / torch.sqrt(mean + eps)
    # relative: the sum's additions, its division, eps, root and reciprocal; halved by the root
    er = rstd * ((_depth(cols) + 4) / 2 + 4) * U32
    y = s * rstd[:, None] * w
    ey = (s * w).abs() * er[:, None] + 3 * U32 * y.abs()
    return (y, rstd), (ey, er)


def rms_backward(dy, x, rstd, w, dsum):
    dt, pdt = x.dtype, x.dtype if w is None else w.dtype
    dy, x = (t.double().cpu().reshape(-1, t.shape[-1]) for t in (dy, x))
    rows, cols = x.shape
    w = torch.ones(cols, dtype=torch.float64) if w is None else w.double().cpu()
    r = rstd.double().cpu().reshape(-1, 1)
    h, g = x * r, dy * w
    c = (g * h).mean(1, keepdim=True)
    dx = r * (g - h * c)
    ec = (_depth(cols) + 6) * U32 * (g * h).abs().mean(1, keepdim=True)
    ex = r * (h.abs() * ec + 6 * U32 * (g.abs() + (h * c).abs()))
    if dsum is not None:
        dsum = dsum.double().cpu().reshape(-1, cols)
        dx = dx + dsum
        ex = ex + U32 * dx.abs()
    dw = (dy * h).sum(0)
    ew = (rows + 6) * U32 * (dy * h).abs().sum(0)
    return (dx, dw), (rounded(dt, dx, ex), rounded(pdt, dw, ew))


# ------------------------------------------------------------------- dropout
def philox(c, k):
    """Philox4x32-10 of counters c (..., 4) and a key (2 words): numpy's unsigned words, multiplied in 64 bits."""
    c = [c[..., i].astype(np.uint64) for i in range(4)]
    k = [int(k[0]), int(k[1])]
    mask = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & mask, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1).astype("<u4")


def kept(rows, cols, p, seed, offset=0, first_row=0, first_col=0):
    """The mask (rows, cols)."""
    blocks = -(-cols // 8)
    c = np.zeros((rows, blocks, 4), dtype=np.uint64)
    c[..., 0] = (np.arange(blocks) + first_col // 8)[None, :]
    c[..., 1] = (np.arange(rows) + first_row)[:, None]
    c[..., 2], c[..., 3] = offset & 0xFFFFFFFF, offset >> 32
    words = philox(c, (seed & 0xFFFFFFFF, seed >> 32))
    return torch.from_numpy((words.view("<u2").reshape(rows, -1)[:, :cols] >= threshold(p)).copy())


def threshold(p):
    return math.floor(p * 65536 + 0.5)


def dropped(x, keep, p, residual=None):
    """y and its bound: one product, one addition, one rounding."""
    dt = x.dtype
    x = x.double().cpu().reshape(keep.shape)
    t = threshold(p)
    y = torch.where(keep, x * (65536 / (65536 - t)) if t < 65536 else x, torch.zeros(()).double())
    e = 2 * U32 * y.abs()
    if residual is not None:
        y = y + residual.double().cpu().reshape(keep.shape)
        e = e + U32 * y.abs()
    return y, rounded(dt, y, e)


# ----------------------------------------------------------------- attention
def _heads(t, heads):
    """(batch, rows, kv heads, d) as (batch, heads, rows, d)."""
    t = t.double().cpu().transpose(1, 2)
    return t.repeat_interleave(heads // t.shape[1], 1)


def _scores(q, k, lengths, scale):
    """Scaled scores, what fp32 may add to them, and which keys exist."""
    h, d = q.shape[2], q.shape[3]
    a, b = _heads(q, h), _heads(k, h).transpose(2, 3)
    s = a @ b * scale
    e = (2 * d + 8) * U32 * (a.abs() @ b.abs()) * scale + 4 * U32 * s.abs()
    there = torch.ones(q.shape[0], 1, 1, k.shape[1], dtype=torch.bool)
    if lengths is not None:
        there = (torch.arange(k.shape[1])[None, :] < lengths.cpu()[:, None])[:, None, None, :]
    return s, e, there


def _clean(t, lengths):
    """``t`` (batch, keys, ..) with zeros in the place of keys that do not exist."""
    t = t.double().cpu()
    if lengths is None:
        return t
    return torch.where((torch.arange(t.shape[1])[None, :] < lengths.cpu()[:, None])[:, :, None, None], t, torch.zeros(()).double())


# P's and dS's roundings for the matrix instructions: half a step, and of values
# below the normal ones half the smallest spacing
P_UNIT = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
P_TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}


def attention(q, k, v, lengths=None, scale=None):
    """(y, lse) and their bounds."""
    dt, h, d = q.dtype, q.shape[2], q.shape[3]
    scale = d ** -0.5 if scale is None else scale
    k, v = _clean(k, lengths), _clean(v, lengths)
    s, es, there = _scores(q, k, lengths, scale)
    n = k.shape[1]
    s = torch.where(there, s, torch.full((), -math.inf).double())
    top = s.amax(-1, keepdim=True) if n else torch.full(s.shape[:3] + (1,), -math.inf).double()
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    # relative error of an exponential: its argument's, one rounding of the difference, the hardware's 2^-22
    ep = es + 4 * U32 * (torch.where(there, (s - top).abs(), torch.zeros_like(es)) + top.abs() + 1)
    total = p.sum(-1, keepdim=True)
    safe = torch.where(total > 0, total, torch.ones_like(total))
    vh = _heads(v, h)
    y = p @ vh / safe
    sums = (2 * n + 8) * U32
    # the running maximum that P is held against may lie 8 bits below the final one, never above: P up to 2^8, its tiny ones relative to 1
    ey = ((p * (ep + P_UNIT[dt] + sums) + P_TINY[dt]) @ vh.abs()) / safe + y.abs() * ((p * ep).sum(-1, keepdim=True) / safe + sums + 4 * U32)
    lse = torch.where(total > 0, top + torch.log(safe), torch.full((), -math.inf).double()).squeeze(-1)
    el = ((p * ep).sum(-1) / safe.squeeze(-1)) + sums + 6 * U32 * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs()) + 4 * U32
    y, ey = (t.transpose(1, 2) for t in (y, rounded(dt, y, ey)))
    return (y, lse), (ey, el)


def attention_backward(dy, q, k, v, y, lse, lengths=None, scale=None):
    """(dq, dk, dv) and their bounds, from the y and lse that are given."""
    dt, h, d = q.dtype, q.shape[2], q.shape[3]
    b, kv, n, rows = q.shape[0], k.shape[2], k.shape[1], q.shape[1]
    scale = d ** -0.5 if scale is None else scale
    k, v = _clean(k, lengths), _clean(v, lengths)
    s, es, there = _scores(q, k, lengths, scale)
    l = lse.double().cpu().unsqueeze(-1)
    safe = torch.where(torch.isinf(l), torch.zeros_like(l), l)
    p = torch.where(there, torch.exp(s - safe), torch.zeros_like(s))
    ep = es + 4 * U32 * ((s - safe).abs() + safe.abs() + 1)
    qh, kh, vh, dyh, yh = (_heads(t, h) for t in (q, k, v, dy, y))
    dp, edp = dyh @ vh.transpose(2, 3), (2 * d + 8) * U32 * (dyh.abs() @ vh.abs().transpose(2, 3))
    delta, edelta = (dyh * yh).sum(-1, keepdim=True), (d + 8) * U32 * (dyh * yh).abs().sum(-1, keepdim=True)
    ds = p * (dp - delta)
    eds = ds.abs() * (ep + 2 * U32) + p * (1 + ep) * (edp + edelta + 2 * U32 * (dp.abs() + delta.abs()))
    eds = torch.where(there, eds + P_UNIT[dt] * (ds.abs() + eds) + P_TINY[dt], torch.zeros_like(eds))
    # fp16 holds P times 2^10
    epv = torch.where(there, p * (ep + P_UNIT[dt] * (1 + ep)) + P_TINY[dt] * 2.0 ** -10, torch.zeros_like(p))
    dq, eq = ds @ kh, eds @ kh.abs() + (2 * n + 8) * U32 * (ds.abs() + eds) @ kh.abs()
    over = (2 * rows * (h // kv) + 8) * U32
    dk, ek = ds.transpose(2, 3) @ qh, (eds + over * (ds.abs() + eds)).transpose(2, 3) @ qh.abs()
    dv, ev = p.transpose(2, 3) @ dyh, (epv + over * (p + epv)).transpose(2, 3) @ dyh.abs()
    shared = lambda t: t.reshape(b, kv, h // kv, n, d).sum(2)  # noqa: E731
    dk, ek, dv, ev = shared(dk) * scale, shared(ek) * scale, shared(dv), shared(ev)
    dq, eq = dq * scale, eq * scale
    out = [(g, rounded(dt, g, e + 2 * U32 * g.abs())) for g, e in ((dq, eq), (dk, ek), (dv, ev))]
    return tuple(g.transpose(1, 2) for g, _ in out), tuple(e.transpose(1, 2) for _, e in out)
