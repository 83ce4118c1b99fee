"""Plain fp64 forms of the block operators, each with a bound on what a
correct kernel may differ by.

The bounds follow from the arithmetic the operators promise: operands exact,
products and sums in fp32 (each addition adds at most one unit roundoff of the
running value, so a sum of n terms is off by at most n u32 sum|terms|; matrix
instructions may round once more per step, hence the factor 2), one rounding
of the output to its type.
"""
import math

import torch

U32 = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# smallest spacing of the type's subnormals (flushed bf16 and fp32 ones: the smallest normal)
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
SLOPE = 1.13          # largest |act'| of the activations here (gelu's 1.129)
CURVE = 1.2           # largest |act''| (the tanh form's 0.80 and a margin)


def act64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    assert name == "sigmoid"
    return torch.sigmoid(z)


def act64_grad(name, z):
    z = z.clone().requires_grad_(True)
    with torch.enable_grad():
        if name == "relu":
            return (z.detach() > 0).double()
        return torch.autograd.grad(act64(name, z).sum(), z)[0]


def act_error(dtype, z):
    """What evaluating an activation (or its slope) in fp32 may add: a few
    roundings, and for the 16-bit types the hardware exponential and
    reciprocal (an argument rounded to fp32 before it: |z| more roundings)."""
    return (2.0 ** -19 if dtype != torch.float32 else 2.0 ** -21) * (1 + z.abs()) ** 2


def mm_error(a, b, k):
    """Of a product a @ b with k terms in fp32."""
    return (2 * k + 8) * U32 * (a.abs() @ b.abs())


def rounded(dtype, v, err):
    return err + UNIT[dtype] * (v.abs() + err) + TINY[dtype]


def linear_forward(x, w, bias, act, residual):
    """(y, pre) and the bounds of both."""
    dt = x.dtype
    x, w = x.double().cpu().reshape(-1, x.shape[-1]), w.double().cpu()
    z, e = x @ w.T, mm_error(x, w.T, x.shape[1])
    if bias is not None:
        z = z + bias.double().cpu()
        e = e + 2 * U32 * z.abs()
    y = act64(act, z)
    ey = e if act == "none" else SLOPE * e + act_error(dt, z)
    if residual is not None:
        y = y + residual.double().cpu().reshape(y.shape)
        ey = ey + U32 * y.abs()
    return (y, z), (rounded(dt, y, ey), rounded(dt, z, e))


def gated_forward(x, w, bias, act):
    dt = x.dtype
    x, w = x.double().cpu().reshape(-1, x.shape[-1]), w.double().cpu()
    n = w.shape[0] // 2
    z, e = x @ w.T, mm_error(x, w.T, x.shape[1])
    if bias is not None:
        z = z + bias.double().cpu()
        e = e + 2 * U32 * z.abs()
    g, u, eg, eu = z[:, :n], z[:, n:], e[:, :n], e[:, n:]
    a = act64(act, g)
    ea = eg if act == "none" else SLOPE * eg + act_error(dt, g)
    y = a * u
    ey = ea * (u.abs() + eu) + a.abs() * eu + U32 * y.abs()
    return (y, z), (rounded(dt, y, ey), rounded(dt, z, e))


def backward(dy, x, w, pre, act, gated):
    """(dx, dw, db) and their bounds; the products read dz rounded to the
    operands' type, the column sums do not."""
    dt = x.dtype
    dy, x, w = dy.double().cpu().reshape(-1, dy.shape[-1]), x.double().cpu().reshape(-1, x.shape[-1]), w.double().cpu()
    if pre is not None:
        pre = pre.double().cpu().reshape(dy.shape[0], -1)
    rows, n = dy.shape
    if gated:
        g, u = pre[:, :n], pre[:, n:]
        a, d = act64(act, g), act64_grad(act, g)
        dz = torch.cat((dy * u * d, dy * a), 1)
        e = torch.cat(((dy * u).abs(), dy.abs()), 1) * torch.cat((act_error(dt, g), act_error(dt, g)), 1) + 4 * U32 * dz.abs()
    elif act != "none":
        dz = dy * act64_grad(act, pre)
        e = dy.abs() * act_error(dt, pre) + 4 * U32 * dz.abs()
    else:
        dz, e = dy, torch.zeros_like(dy)
    ez = rounded(dt, dz, e) if gated or act != "none" else e
    dx, dw, db = dz @ w, dz.T @ x, dz.sum(0)
    bx = rounded(dt, dx, ez @ w.abs() + mm_error(dz.abs() + ez, w, dz.shape[1]))
    bw = rounded(dt, dw, ez.T @ x.abs() + mm_error((dz.abs() + ez).T, x, rows))
    bb = rounded(dt, db, e.sum(0) + rows * U32 * (dz.abs() + e).sum(0))
    return (dx, dw, db), (bx, bw, bb)


def _depth(cols):
    """Additions in a row in a row's sums: what a thread adds up, and the tree over threads and waves."""
    return 64 + cols / 1024


def norm_forward(x, w, b, eps):
    dt = x.dtype
    x = x.double().cpu().reshape(-1, x.shape[-1])
    cols = x.shape[1]
    w = torch.ones(cols, dtype=torch.float64) if w is None else w.double().cpu()
    b = torch.zeros(cols, dtype=torch.float64) if b is None else b.double().cpu()
    mean = x.mean(1)
    c = x - mean[:, None]
    var = (c * c).mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    y = c * rstd[:, None] * w + b
    em = _depth(cols) * U32 * x.abs().mean(1) + 2 * U32 * mean.abs()
    ec = em[:, None] + 2 * U32 * (x.abs() + mean.abs()[:, None])
    ev = (2 * c.abs() * ec + ec * ec).mean(1) + (_depth(cols) + 4) * U32 * var
    er = rstd * torch.clamp(ev / (2 * (var + eps)) * 1.5 + 6 * U32, max=1e30)
    ey = w.abs() * (ec * (rstd + er)[:, None] + c.abs() * er[:, None]) + 3 * U32 * ((c * rstd[:, None] * w).abs() + b.abs())
    return (y, mean, rstd), (rounded(dt, y, ey), em + TINY[torch.float32], er)


def norm_backward(dy, x, mean, rstd, w):
    dt, pdt = x.dtype, x.dtype if w is None else w.dtype
    dy, x = (t.double().cpu().reshape(-1, t.shape[-1]) for t in (dy, x))
    rows, cols = x.shape
    w = torch.ones(cols, dtype=torch.float64) if w is None else w.double().cpu()
    m, r = mean.double().cpu().reshape(-1, 1), rstd.double().cpu().reshape(-1, 1)
    h = (x - m) * r
    eh = 3 * U32 * (x.abs() + m.abs()) * r
    g = dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = r * (g - c1 - h * c2)
    n = _depth(cols) + 4
    e1 = n * U32 * g.abs().mean(1, keepdim=True)
    e2 = n * U32 * (g * h).abs().mean(1, keepdim=True) + (g.abs() * eh).mean(1, keepdim=True)
    ex = r * (e1 + h.abs() * e2 + eh * (c2.abs() + e2) + 6 * U32 * (g.abs() + c1.abs() + (h * c2).abs()))
    dw, db = (dy * h).sum(0), dy.sum(0)
    ew = (dy.abs() * eh).sum(0) + (rows + 4) * U32 * (dy * h).abs().sum(0)
    eb = (rows + 4) * U32 * dy.abs().sum(0)
    return (dx, dw, db), (rounded(dt, dx, ex), rounded(pdt, dw, ew), rounded(pdt, db, eb))


def assert_within(got, want, bound, what):
    got = got.detach().double().cpu().reshape(want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = int(torch.argmax((off / bound).nan_to_num(nan=float("inf")).flatten()))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds; worst at {i}: got "
                             f"{got.flatten()[i].item()}, want {want.flatten()[i].item()} +- {bound.flatten()[i].item()}")
