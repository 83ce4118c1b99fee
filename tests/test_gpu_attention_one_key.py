"""Gradients of rows with one key: P is 1 and dS = dP - delta is 0, so dq and dk
are the rounding of two fp32 sums, which no relative error can judge.

Their bound: y is the key's v up to three roundings in fp32, e v, 1 / e and their
product, with e = exp(s - m) near 1: 3 x 2^-24 and terms of 2^-48, taken as 4 x
2^-24 (the 16-bit types' last rounding removes it).  dP and delta are fp32 sums of
d terms dy v and dy y, each off by at most d 2^-24 sum |dy v|, and apart by y's
4 x 2^-24 of it; dS is off by all three, and its rounding to the operands' type
adds a part of 2^-8 at most.  dq = scale dS k, and
dk adds scale dS q over the query rows that share the key."""
import pytest
import torch

import ring_allreduce_reduce_amd as ra

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("b, lq, h, kv, d", [(12, 6, 8, 2, 128), (3, 130, 4, 4, 64), (2, 1, 7, 1, 40)])
def test_one_key(b, lq, h, kv, d, dtype):
    gen = torch.Generator().manual_seed(b + lq)
    q, k, v, dy = (torch.randn(*s, generator=gen).to(dtype).cuda() for s in ((b, lq, h, d), (b, 1, kv, d), (b, 1, kv, d), (b, lq, h, d)))
    y, lse = ra.cross_attention(q, k, v, stats=True)
    dq, dk, dv = ra.cross_attention_backward(dy, q, k, v, y, lse)
    Q, K, V, DY = (t.double() for t in (q, k, v, dy))
    K, V = (t.repeat_interleave(h // kv, 2) for t in (K, V))
    off = 4 * 2.0 ** -24 if dtype == torch.float32 else 0.0
    assert ((y.double() - V).abs() <= off * V.abs()).all()
    ds = (2 * d + 4) * 2.0 ** -24 * (1 + 2.0 ** -8) * (DY * V).abs().sum(-1, keepdim=True) * d ** -0.5
    assert (dq.double().abs() <= ds * K.abs() * (1 + 2.0 ** -8)).all()
    most = (ds * Q.abs()).reshape(b, lq, kv, h // kv, d).sum((1, 3))[:, None] * (1 + 2.0 ** -8)
    assert (dk.double().abs() <= most).all()
    exact = DY.reshape(b, lq, kv, h // kv, d).sum((1, 3))[:, None]
    # P: 1 up to lse's rounding and the exponential's; then sums of lq group terms and one rounding
    far = (torch.finfo(dtype).eps + 2.0 ** -18 + lq * (h // kv) * 2.0 ** -24) * DY.abs().reshape(b, lq, kv, h // kv, d).sum((1, 3))[:, None]
    assert ((dv.double() - exact).abs() <= far).all()
