"""A tensor-parallel feed-forward block over virtual ranks, forward and backward.

    y = x + AllReduce_r(W_down,r (act(W_gate,r n) * (W_up,r n))) + b,   n = LayerNorm(x)

Every rank holds a share of the hidden width: its gate and up rows, and the
matching columns of the down projection.  The ranks' partial outputs are added
by the AllReduce (rank 0's epilogue brings the bias and the residual), and so
are their partial gradients of n on the way back.

    python -m ring_allreduce_reduce_amd.examples.tensor_parallel_block [--ranks 4] [--rows 2048] ...

prints how far the sharded block is from the same block in fp32 on one rank,
and the time of a step.
"""
from __future__ import annotations

import argparse

import torch

import ring_allreduce_reduce_amd as ra


class Block:
    """One block's parameters, split over ``ranks``."""

    def __init__(self, ranks, width, hidden, dtype=torch.bfloat16, act="silu", seed=0):
        if hidden % ranks:
            raise ValueError("the hidden width must divide over the ranks")
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)

        share = hidden // ranks
        self.ranks, self.act = ranks, act
        self.norm_weight, self.norm_bias = 1 + normal(width, scale=0.1), normal(width, scale=0.1)
        # the gate's rows and then the up projection's, and the down projection's columns
        self.gate_up = [normal(2 * share, width, scale=width ** -0.5) for _ in range(ranks)]
        self.down = [normal(width, share, scale=hidden ** -0.5) for _ in range(ranks)]
        self.bias = normal(width, scale=0.1)

    def forward(self, x):
        """(y, what the backward pass needs)."""
        n, mean, rstd = ra.layer_norm(x, self.norm_weight, self.norm_bias, stats=True)
        kept, parts = [], []
        for r in range(self.ranks):
            h, pre = ra.gated_ffn(n, self.gate_up[r], act=self.act, save_pre=True)
            first = r == 0
            parts.append(ra.linear(h, self.down[r], self.bias if first else None, residual=x if first else None))
            kept.append((h, pre))
        ra.allreduce(parts, parts, op="sum")
        return parts[0], (x, n, mean, rstd, kept)

    def backward(self, dy, saved):
        """Gradients of x and of every parameter (the ranks' shares as lists)."""
        x, n, mean, rstd, kept = saved
        d_gate_up, d_down, parts, d_bias = [], [], [], None
        for r, (h, pre) in enumerate(kept):
            dh, dw, db = ra.linear_backward(dy, h, self.down[r], dbias=r == 0)
            d_bias = db if r == 0 else d_bias
            dn, dgu, _ = ra.gated_ffn_backward(dh, n, self.gate_up[r], pre, act=self.act, dbias=False)
            d_down.append(dw)
            d_gate_up.append(dgu)
            parts.append(dn)
        ra.allreduce(parts, parts, op="sum")
        dx, d_weight, d_norm_bias = ra.layer_norm_backward(parts[0], x, mean, rstd, self.norm_weight)
        return {"x": dx + dy, "norm_weight": d_weight, "norm_bias": d_norm_bias, "gate_up": d_gate_up, "down": d_down,
                "bias": d_bias}

    def plain(self, x, dy):
        """The unsharded block in fp32 through torch's own differentiation:
        (y, gradients named as backward's)."""
        f = lambda t: t.float().requires_grad_(True)  # noqa: E731
        x, w, b, bias = f(x), f(self.norm_weight), f(self.norm_bias), f(self.bias)
        gate_up, down = [f(t) for t in self.gate_up], [f(t) for t in self.down]
        n = (x - x.mean(-1, keepdim=True)) * (x.var(-1, unbiased=False, keepdim=True) + 1e-5).rsqrt() * w + b
        y = x + bias
        for gu, d in zip(gate_up, down):
            g, u = (n @ gu.t()).chunk(2, -1)
            y = y + (g * torch.sigmoid(g) * u) @ d.t()
        leaves = [x, w, b, bias, *gate_up, *down]
        g = torch.autograd.grad(y, leaves, dy.float())
        r = self.ranks
        return y.detach(), {"x": g[0], "norm_weight": g[1], "norm_bias": g[2], "bias": g[3], "gate_up": list(g[4:4 + r]),
                            "down": list(g[4 + r:])}


def distance(got, want):
    """Relative distance of tensors, or of lists of them."""
    if isinstance(want, (list, tuple)):
        return max(distance(a, b) for a, b in zip(got, want))
    return float((got.float() - want).norm() / want.norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    block = Block(a.ranks, a.width, a.hidden)
    x = torch.randn(a.rows, a.width, device="cuda").to(torch.bfloat16)
    dy = (0.1 * torch.randn(a.rows, a.width, device="cuda")).to(torch.bfloat16)
    y, saved = block.forward(x)
    grads = block.backward(dy, saved)
    torch.cuda.synchronize()
    want, plain = block.plain(x, dy)
    print(f"y: {distance(y, want):.2e} from fp32; gradients: " + ", ".join(f"{k} {distance(grads[k], plain[k]):.2e}" for k in grads))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        block.backward(dy, block.forward(x)[1])
    end.record()
    torch.cuda.synchronize()
    ms = begin.elapsed_time(end) / a.steps
    flops = 18 * a.rows * a.width * a.hidden          # three products forward, six backward
    print(f"{a.ranks} ranks, {a.rows} rows, {a.width} x {a.hidden}: {ms:.3f} ms a step, {flops / ms / 1e9:.0f} TFLOP/s")
    code = ra.ringar_get_async_error(torch.cuda.current_stream().cuda_stream)
    if code != ra.SUCCESS:
        raise ra.RingarError(code, "allreduce")


if __name__ == "__main__":
    main()
