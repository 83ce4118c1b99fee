"""Attention's gradients where P times dy is small, or dy rises or falls over many
powers of two: fp16 holds dS = P (dP - delta) times a power of two.

The bound: a dS is off by half a step of fp16, 2^-11 of its value, or by what the
type's smallest step, 2^-24, leaves: 2^-25 at 2^up times dS.  dq's power puts the
row's largest |dP - delta| of the first 32 keys beyond 2^9, so that is 2^-34 of it
(where a later one overflows, 2^10 times that; where it overflows again, 2^-25 at dS's
natural size); dk's puts the largest dS of 32 keys beyond 2^9: 2^-34 of it."""
import zlib

import pytest
import torch

import layer_refs as L
import ring_allreduce_reduce_amd as ra
from block_refs import U32, assert_within, rounded

pytestmark = pytest.mark.gpu
F16 = torch.float16


def _gen(*key):
    print("case", *key, flush=True)
    g = torch.Generator()
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def _rand(g, *shape):
    return torch.randn(shape, generator=g)


def _check(dy, q, k, v, scale, tiny_q=lambda away: 2.0 ** -34 * away.amax(-1, keepdim=True), lengths=None):
    """Kernel's dq and dk within the bound; tiny_q: what the smallest step leaves of a dS, from |dP - delta|."""
    y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, scale=scale, stats=True)
    grads = ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths, scale=scale)
    b, rows, h, d = q.shape
    n, kv = k.shape[1:3]
    s, es, there = L._scores(q, k, lengths, scale)
    l = lse.double().cpu().unsqueeze(-1)
    p = torch.where(there, torch.exp(s - l), torch.zeros_like(s))
    ep = es + 4 * U32 * ((s - l).abs() + l.abs() + 1)
    qh, kh, vh, dyh, yh = (L._heads(t, h) for t in (q, k, v, dy, y))
    dp, edp = dyh @ vh.transpose(2, 3), (2 * d + 8) * U32 * (dyh.abs() @ vh.abs().transpose(2, 3))
    delta, edelta = (dyh * yh).sum(-1, keepdim=True), (d + 8) * U32 * (dyh * yh).abs().sum(-1, keepdim=True)
    ds = p * (dp - delta)
    e32 = ds.abs() * (ep + 2 * U32) + p * (1 + ep) * (edp + edelta + 2 * U32 * (dp.abs() + delta.abs()))
    unit = L.P_UNIT[q.dtype]
    away = torch.where(there, (dp - delta).abs(), torch.zeros_like(dp))
    most_k = ds.abs().reshape(b, kv, -1).amax(-1).repeat_interleave(h // kv, 1)[:, :, None, None]
    eq, ek = (torch.where(there, e32 + unit * (ds.abs() + e32) + t, torch.zeros_like(ds)) for t in (tiny_q(away), 2.0 ** -34 * most_k))
    dq, off_q = ds @ kh, (eq + (2 * n + 8) * U32 * (ds.abs() + eq)) @ kh.abs()
    over = (2 * rows * (h // kv) + 8) * U32
    dk, off_k = ds.transpose(2, 3) @ qh, (ek + over * (ds.abs() + ek)).transpose(2, 3) @ qh.abs()
    dk, off_k = (t.reshape(b, kv, h // kv, n, d).sum(2) for t in (dk, off_k))
    for got, want, off, what in ((grads[0], dq * scale, off_q * scale, "dq"), (grads[1], dk * scale, off_k * scale, "dk")):
        off = rounded(q.dtype, want, off + 2 * U32 * want.abs())
        assert_within(got, want.transpose(1, 2), off.transpose(1, 2), what)
    return grads


SIZES = [(1, 70, 2048, 4, 2, 64), (2, 33, 300, 2, 2, 128), (1, 1, 1500, 8, 2, 80), (3, 130, 96, 2, 1, 40), (1, 200, 5000, 1, 1, 128)]


@pytest.mark.parametrize("times", [2.0 ** -7, 2.0 ** -10, 2.0 ** -14])
@pytest.mark.parametrize("wide", ["q", "k"])
@pytest.mark.parametrize("b,lq,n,h,kv,d", SIZES)
def test_small_dy(b, lq, n, h, kv, d, wide, times):
    """Large keys (dq, then, is no subnormal number) or large queries (dk)."""
    g = _gen("small", b, lq, n, d, wide, times)
    q, k, v, dy = _rand(g, b, lq, h, d), _rand(g, b, n, kv, d), _rand(g, b, n, kv, d), _rand(g, b, lq, h, d) * times
    large, small = 64.0, d ** -0.5 / 64
    q, k = (q * large, k * small) if wide == "q" else (q * small, k * large)
    _check(*(t.to(F16).cuda() for t in (dy, q, k, v)), 1.0)


@pytest.mark.parametrize("b,lq,n,h,kv,d", SIZES)
def test_rows_of_unlike_size(b, lq, n, h, kv, d):
    """dy of neighbouring rows 2^7 apart, some of them zero; ragged lengths."""
    g = _gen("unlike", b, lq, n, d)
    q, k, v, dy = _rand(g, b, lq, h, d) * 64, _rand(g, b, n, kv, d) * d ** -0.5, _rand(g, b, n, kv, d), _rand(g, b, lq, h, d)
    size = torch.tensor([1.0, 2.0 ** -7, 0.0, 2.0 ** -14])[torch.arange(lq) % 4]
    dy = (dy * size[None, :, None, None]).to(F16).cuda()
    lengths = torch.tensor([n - i * n // 3 for i in range(b)], dtype=torch.int32, device="cuda")
    grads = _check(dy, *(t.to(F16).cuda() for t in (q, k, v)), 1.0 / 64, lengths=lengths)
    assert (grads[0][:, size == 0] == 0).all()


@pytest.mark.parametrize("b,lq,n,h,kv,d", SIZES)
def test_dy_beyond_what_the_type_holds_of_ds(b, lq, n, h, kv, d):
    """|dP| near 2^28 and P near 1 / n: dS at its natural size would be infinite in fp16."""
    g = _gen("large", b, lq, n, d)
    q, k, v, dy = _rand(g, b, lq, h, d) * 2.0 ** -8, _rand(g, b, n, kv, d) * 2.0 ** -12, _rand(g, b, n, kv, d) * 4096, _rand(g, b, lq, h, d) * 8192
    grads = _check(*(t.to(F16).cuda() for t in (dy, q, k, v)), 2.0 ** -5)
    assert all(t.isfinite().all() for t in grads[:2])


@pytest.mark.parametrize("base,far,times", [(1.0, 512.0, 0.25), (2.0 ** -4, 4096.0, 0.25), (2.0 ** -8, 4096.0, 0.125)])
@pytest.mark.parametrize("b,lq,n,h,kv,d", [s for s in SIZES if s[2] > 40])
def test_values_far_beyond_those_of_the_first_keys(b, lq, n, h, kv, d, base, far, times):
    """The last keys have values 2^9, 2^16 or 2^20 times the others', one the negative of the other, and half of
    the rows give each a third of their weight, so that delta stays small: dS overflows at the first power, and at the
    second one for the largest."""
    g = _gen("outlier", b, lq, n, d, base)
    q, k, v, dy = _rand(g, b, lq, h, d), _rand(g, b, n, kv, d), _rand(g, b, n, kv, d) * base, _rand(g, b, lq, h, d) * times
    v[:, -1] = _rand(g, b, kv, d).sign() * far
    v[:, -2] = -v[:, -1]
    q[..., 0] = (torch.arange(lq) % 2 * d ** 0.5)[None, :, None]
    k[..., 0] = 0.0
    k[:, -2:, :, 1:] = 0.0
    k[:, -2:, :, 0] = torch.tensor(float(n)).log() + 0.5

    def tiny(away):
        return torch.clamp(2.0 ** -24 * away[..., :-2].amax(-1, keepdim=True), min=2.0 ** -25)
    _check(*(t.to(F16).cuda() for t in (dy, q, k, v)), d ** -0.5, tiny_q=tiny)


def test_nan_in_dy_stays_in_its_row():
    g = _gen("nan")
    q, k, v, dy = (t.to(F16).cuda() for t in (_rand(g, 2, 50, 4, 64), _rand(g, 2, 700, 4, 64), _rand(g, 2, 700, 4, 64), _rand(g, 2, 50, 4, 64) * 2.0 ** -12))
    y, lse = ra.cross_attention(q, k, v, stats=True)
    want = ra.cross_attention_backward(dy, q, k, v, y, lse)
    for bad in (float("nan"), float("inf")):
        d2 = dy.clone()
        d2[1, 3, 2, 5] = bad
        dq, dk, dv = ra.cross_attention_backward(d2, q, k, v, y, lse)
        assert not dq[1, 3, 2].isfinite().any()
        same = torch.ones_like(dq, dtype=torch.bool)
        same[1, 3, 2] = False
        assert torch.equal(dq[same], want[0][same])
        heads = [i for i in range(4) if i != 2]
        assert torch.equal(dk[:, :, heads], want[1][:, :, heads]) and torch.equal(dk[0], want[1][0])
        assert not dk[1, :, 2].isfinite().any()
