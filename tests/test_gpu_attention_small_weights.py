"""Attention where most keys have weights near 2^-24 of one key's, and that one's
value is small: what the many leave must keep the type's precision.  In fp16 these
weights are below the type's normal numbers unless P is held above them.

The bound: P is held so that the first tile's largest is 2^10 (a later tile's, once one
has passed 65504, 2^4), so it is off by half a step of its own, 2^-11 of it, or by
2^-25 2^-10 (2^-25 2^-4) of the largest; the rest as elsewhere (layer_refs)."""
import zlib

import pytest
import torch

import layer_refs as L
import ring_allreduce_reduce_amd as ra
from block_refs import U32, assert_within, rounded

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TINY = {F32: 0.0, F16: 2.0 ** -35, BF16: 2.0 ** -126}


def _check(q, k, v, raised=False):
    """y within the bound, in fp64 on the GPU (some hundred thousand keys)."""
    dt, h, d = q.dtype, q.shape[2], q.shape[3]
    y, lse = ra.cross_attention(q, k, v, stats=True)
    heads = lambda t: t.double().transpose(1, 2).repeat_interleave(h // t.shape[2], 1).contiguous()  # noqa: E731
    qh, kh, vh = heads(q), heads(k), heads(v)
    kt, n = kh.transpose(2, 3).contiguous(), k.shape[1]
    s = torch.matmul(qh, kt) * d ** -0.5
    es = (2 * d + 8) * U32 * torch.matmul(qh.abs(), kt.abs()) * d ** -0.5 + 4 * U32 * s.abs()
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    ep = es + 4 * U32 * ((s - top).abs() + top.abs() + 1)
    total = p.sum(-1, keepdim=True)
    want = torch.matmul(p, vh) / total
    sums = (2 * n + 8) * U32
    tiny = TINY[dt] * (2.0 ** 6 if raised else 1)
    off = torch.matmul(p * (ep + L.P_UNIT[dt] + sums) + tiny, vh.abs()) / total + want.abs() * ((p * ep).sum(-1, keepdim=True) / total + sums + 4 * U32)
    assert_within(y, want.transpose(1, 2).cpu(), rounded(dt, want, off).transpose(1, 2).cpu(), "y")
    l = (top + torch.log(total)).squeeze(-1)
    assert ((lse.double() - l).abs() <= (p * ep).sum(-1) / total.squeeze(-1) + sums + 6 * U32 * l.abs() + 4 * U32).all()


def _operands(dtype, b, lq, n, h, d, sink, bits):
    """Scores of 0 and, at key `sink`, bits ln 2 (a little off, so that the many are no power of two of it)."""
    print("case", dtype, b, lq, n, h, d, sink, bits, flush=True)
    g = torch.Generator().manual_seed(zlib.crc32(repr((b, lq, n, h, d, sink, bits)).encode()))
    q, k = torch.zeros(b, lq, h, d), torch.zeros(b, n, h, d)
    q[..., 0] = 1.0
    k[:, sink, :, 0] = (bits - 0.4) * 0.6931 * d ** 0.5
    v = 1.0 + 0.25 * torch.randn(b, n, h, d, generator=g)
    v[:, sink] = 0.0
    return [t.to(dtype).cuda() for t in (q, k, v)]


# one token, keys in parts; 32 rows and all keys in one part; blocks of 128 rows
SIZES = [(1, 1, 100003, 2, 64), (1, 1, 40000, 2, 128), (8, 20, 4001, 40, 64), (2, 150, 5000, 8, 64), (2, 257, 3001, 16, 128)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("bits", [12, 20, 24])
@pytest.mark.parametrize("b,lq,n,h,d", SIZES)
def test_the_first_key_outweighs_the_others(b, lq, n, h, d, bits, dtype):
    _check(*_operands(dtype, b, lq, n, h, d, 0, bits))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("bits", [7, 12, 20])
@pytest.mark.parametrize("b,lq,n,h,d", SIZES)
def test_a_later_key_outweighs_the_others(b, lq, n, h, d, bits, dtype):
    _check(*_operands(dtype, b, lq, n, h, d, n // 2, bits), raised=True)


@pytest.mark.parametrize("b,lq,n,h,d", SIZES)
def test_like_scores(b, lq, n, h, d):
    """As large a sum of a tile as scores without a larger one can give."""
    q, k, v = _operands(F16, b, lq, n, h, d, 0, 0.4)
    v[:, 0] = 1.0
    _check(q, k, v)
