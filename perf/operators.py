"""What the tensor-parallel block's operators are measured on: layer norm, the
linear product with its epilogue, and the gated feed-forward, each forward and
backward, from one token to a training step's batch.

``run`` computes a case in its plain form (elementary torch operations in
fp32, rounded once at the end), or with ``own`` set through the package's
operators; ``exact`` gives the same outputs in fp64.
"""
import math

import torch

own = False

TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
BYTES = {"float32": 4, "float16": 2, "bfloat16": 2}
EPS = 1e-5


def listed():
    return [
        # a decoding step's norm before a projection: one token
        dict(name="norm_token", op="layer_norm", direction="forward", dtype="bfloat16", rows=1, cols=4096, train=False),
        # a training step's norm, statistics kept for the backward pass
        dict(name="norm_train", op="layer_norm", direction="forward", dtype="bfloat16", rows=16384, cols=8192, train=True),
        # a small fp32 model's norm, with rows that do not divide and an odd width
        dict(name="norm_back_odd", op="layer_norm", direction="backward", dtype="float32", rows=2053, cols=1001, train=True),
        # a training step's norm backward with both parameter gradients
        dict(name="norm_back", op="layer_norm", direction="backward", dtype="bfloat16", rows=16384, cols=4096, train=True),
        # one token through an output projection, bias and residual added
        dict(name="linear_token", op="linear", direction="forward", dtype="bfloat16", rows=1, inner=4096, outer=4096,
             act="none", bias=True, residual=True, train=False),
        # a prompt of odd length through a layer whose widths are odd too
        dict(name="linear_odd", op="linear", direction="forward", dtype="float16", rows=333, inner=1023, outer=2049,
             act="gelu", bias=True, residual=True, train=False),
        # a training step's expanding layer, pre-activation kept
        dict(name="linear_train", op="linear", direction="forward", dtype="bfloat16", rows=8192, inner=4096, outer=16384,
             act="gelu_tanh", bias=True, residual=False, train=True),
        # its backward pass: three gradients
        dict(name="linear_back", op="linear", direction="backward", dtype="bfloat16", rows=4096, inner=4096, outer=16384,
             act="gelu_tanh", bias=True, residual=False, train=True),
        # a batch of decoding sequences through a rank's share of the gated block
        dict(name="gated_tokens", op="gated_ffn", direction="forward", dtype="bfloat16", rows=16, inner=4096, outer=10240,
             act="silu", bias=False, residual=False, train=False),
        # a prompt's tokens through it
        dict(name="gated_prompt", op="gated_ffn", direction="forward", dtype="bfloat16", rows=2500, inner=4096, outer=10240,
             act="silu", bias=False, residual=False, train=False),
        # a small fp32 model's backward pass
        dict(name="gated_back_fp32", op="gated_ffn", direction="backward", dtype="float32", rows=1000, inner=1024, outer=2736,
             act="gelu", bias=True, residual=False, train=True),
        # a training step's backward pass
        dict(name="gated_back", op="gated_ffn", direction="backward", dtype="bfloat16", rows=8192, inner=4096, outer=10240,
             act="silu", bias=False, residual=False, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: mostly a multiple of 8, 64 or 128, as layers have it, at times any
    odd number; always an odd multiple, so that tiles end inside it."""
    step = rng.choice((1, 8, 64, 128, 128))
    return (_log(rng, lo, hi) // step | 1) * step


def draw(rng):
    op = rng.choice(("layer_norm", "linear", "linear", "gated_ffn", "gated_ffn"))
    direction = rng.choice(("forward", "backward"))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
    train = direction == "backward" or rng.random() < 0.4
    if op == "layer_norm":
        while True:
            case = dict(op=op, direction=direction, dtype=dtype, rows=_log(rng, 1, 16384), cols=_width(rng, 64, 16384), train=train)
            if case["rows"] * case["cols"] <= 1 << 27:
                return case
    while True:
        case = dict(op=op, direction=direction, dtype=dtype, rows=_log(rng, 1, 8192), inner=_width(rng, 64, 8192),
                    outer=_width(rng, 64, 16384), act=rng.choice(("silu", "gelu", "gelu_tanh", "relu")),
                    bias=rng.random() < 0.5, residual=op == "linear" and direction == "forward" and rng.random() < 0.5, train=train)
        if op == "linear" and rng.random() < 0.3:
            case["act"] = "none"
        if work(case)["flops"] <= 1e12 and case["rows"] * case["outer"] <= 1 << 27:
            return case


def work(case):
    m, size = case["rows"], BYTES[case["dtype"]]
    if case["op"] == "layer_norm":
        d = case["cols"]
        if case["direction"] == "forward":
            return {"bytes": (2 * m * d + 2 * d) * size + (8 * m if case["train"] else 0), "flops": 8 * m * d}
        return {"bytes": (3 * m * d + 3 * d) * size + 8 * m, "flops": 14 * m * d}
    k, n = case["inner"], case["outer"]
    gated = case["op"] == "gated_ffn"
    wide = 2 * n if gated else n
    bias = wide if case["bias"] else 0
    if case["direction"] == "forward":
        moved = m * k + wide * k + bias + m * n + (m * n if case["residual"] else 0) + (m * wide if case["train"] else 0)
        return {"bytes": moved * size, "flops": 2 * m * wide * k}
    pre = m * wide if gated or case["act"] != "none" else 0
    moved = m * n + pre + m * k + wide * k + m * k + wide * k + bias
    return {"bytes": moved * size, "flops": 4 * m * wide * k}


def _normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, m = TYPES[case["dtype"]], case["rows"]
    if case["op"] == "layer_norm":
        d = case["cols"]
        # a residual stream: channels of unlike scale and mean
        x = (_normal(gen, m, d) * (0.5 + _normal(gen, 1, d).abs()) + 0.3 * _normal(gen, 1, d)).to(dt)
        state = dict(case=case, x=x, weight=(1 + _normal(gen, d, scale=0.1)).to(dt), bias=_normal(gen, d, scale=0.1, dtype=dt))
        if case["direction"] == "backward":
            state["dy"] = _normal(gen, m, d, dtype=dt)
            x32 = x.float()
            state["mean"] = x32.mean(-1)
            state["rstd"] = (x32.var(-1, unbiased=False) + EPS).rsqrt()
        return state
    k, n = case["inner"], case["outer"]
    wide = 2 * n if case["op"] == "gated_ffn" else n
    state = dict(case=case, x=_normal(gen, m, k, dtype=dt), weight=_normal(gen, wide, k, scale=k ** -0.5, dtype=dt),
                 bias=_normal(gen, wide, scale=0.1, dtype=dt) if case["bias"] else None,
                 residual=_normal(gen, m, n, dtype=dt) if case["residual"] else None)
    if case["direction"] == "backward":
        state["dy"] = _normal(gen, m, n, scale=0.1, dtype=dt)
        # what the forward pass kept: products of unit variance
        state["pre"] = _normal(gen, m, wide, dtype=dt) if wide > n or case["act"] != "none" else None
    return state


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z * torch.sigmoid(z)


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def _plain(state):
    case, x, dt = state["case"], state["x"].float(), state["x"].dtype
    if case["op"] == "layer_norm":
        w = state["weight"].float()
        if case["direction"] == "forward":
            mean = x.mean(-1)
            c = x - mean[:, None]
            rstd = ((c * c).mean(-1) + EPS).rsqrt()
            y = (c * rstd[:, None] * w + state["bias"].float()).to(dt)
            return (y, mean, rstd) if case["train"] else y
        dy, rstd = state["dy"].float(), state["rstd"][:, None]
        h = (x - state["mean"][:, None]) * rstd
        g = dy * w
        dx = rstd * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
        return dx.to(dt), (dy * h).sum(0).to(dt), dy.sum(0).to(dt)
    w, act, n = state["weight"].float(), case["act"], case["outer"]
    if case["direction"] == "forward":
        z = x @ w.t()
        if case["bias"]:
            z = z + state["bias"].float()
        if case["op"] == "gated_ffn":
            y = _act(act, z[:, :n]) * z[:, n:]
        else:
            y = _act(act, z)
            if case["residual"]:
                y = y + state["residual"].float()
        return (y.to(dt), z.to(dt)) if case["train"] else y.to(dt)
    dz = state["dy"].float()
    if case["op"] == "gated_ffn":
        gate, up = state["pre"][:, :n].float(), state["pre"][:, n:].float()
        dz = torch.cat((dz * up * _act_grad(act, gate), dz * _act(act, gate)), 1)
    elif act != "none":
        dz = dz * _act_grad(act, state["pre"].float())
    grads = [(dz @ w).to(dt), (dz.t() @ x).to(dt)]
    if case["bias"]:
        grads.append(dz.sum(0).to(dt))
    return grads


def _kernels(state):
    import ring_allreduce_reduce_amd as ra

    case, x, w = state["case"], state["x"], state["weight"]
    if case["op"] == "layer_norm":
        if case["direction"] == "forward":
            return ra.layer_norm(x, w, state["bias"], EPS, stats=case["train"])
        return ra.layer_norm_backward(state["dy"], x, state["mean"], state["rstd"], w)
    if case["direction"] == "forward":
        if case["op"] == "gated_ffn":
            return ra.gated_ffn(x, w, state["bias"], act=case["act"], save_pre=case["train"])
        return ra.linear(x, w, state["bias"], act=case["act"], residual=state["residual"], save_pre=case["train"])
    back = ra.gated_ffn_backward if case["op"] == "gated_ffn" else ra.linear_backward
    grads = back(state["dy"], x, w, state["pre"], act=case["act"], dbias=case["bias"])
    return list(grads if case["bias"] else grads[:2])


def run(state):
    return _kernels(state) if own else _plain(state)


def exact(case, seed):
    """The outputs in fp64: the forward pass from its definition, gradients by differentiating it."""
    state = prepare(case, seed)
    d = {k: v.double() for k, v in state.items() if isinstance(v, torch.Tensor)}
    x, w = d["x"], d["weight"]
    if case["op"] == "layer_norm":
        leaves = [x, w, d["bias"]]
        for t in leaves:
            t.requires_grad_(case["direction"] == "backward")
        mean = x.mean(-1, keepdim=True)
        var = (x * x).mean(-1, keepdim=True) - mean * mean
        y = (x - mean) / torch.sqrt(var + EPS) * w + d["bias"]
        if case["direction"] == "backward":
            return torch.autograd.grad(y, leaves, d["dy"])
        return (y, mean.squeeze(-1), 1 / torch.sqrt(var + EPS).squeeze(-1)) if case["train"] else y

    def activated(z):
        """The layer's output of its pre-activation."""
        gate = z[:, :case["outer"]]
        name = case["act"]
        if name == "relu":
            a = torch.where(gate > 0, gate, torch.zeros_like(gate))
        elif name == "gelu":
            a = gate * torch.special.ndtr(gate)
        elif name == "gelu_tanh":
            a = gate / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)))
        elif name == "silu":
            a = gate / (1 + torch.exp(-gate))
        else:
            a = gate
        return a * z[:, case["outer"]:] if case["op"] == "gated_ffn" else a

    if case["direction"] == "forward":
        z = torch.mm(x, w.t())
        if case["bias"]:
            z = z + d["bias"]
        y = activated(z)
        if case["residual"]:
            y = d["residual"] + y
        return (y, z) if case["train"] else y
    if "pre" in d:
        pre = d["pre"].requires_grad_(True)
        dz = torch.autograd.grad(activated(pre), pre, d["dy"])[0]
    else:
        dz = d["dy"]
    out = [torch.mm(dz, w), torch.mm(dz.t(), x)]
    if case["bias"]:
        out.append(torch.mm(torch.ones(1, dz.shape[0], dtype=dz.dtype, device=dz.device), dz)[0])
    return out
