"""Attention at the ends of its ranges: every head_dim, keys and queries that lie more
than 2^32 bytes apart within a sequence, some ten thousand sequences, more keys than
2^20."""
import pytest
import torch

import layer_refs as L
import ring_allreduce_reduce_amd as ra
from block_refs import assert_within
from test_gpu_attention import _check, _gen, _lengths

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_every_head_dim(dtype):
    each = 4 if dtype == F32 else 8
    for d in range(each, 129, each):
        _check(_gen("dim", d, dtype), dtype, 2, 9, 70, 2, 1, d, lengths=_lengths(70, 33))


def test_keys_and_queries_beyond_32_bits_of_bytes():
    """200003 keys and 150001 queries, 2^15 bytes from each other."""
    print("case far rows", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    pitch, d = 1 << 14, 64

    def far(rows, at, big=[]):
        if not big:
            big.append(torch.zeros(200003 * pitch, dtype=BF16, device="cuda"))
        t = big[0].as_strided((1, rows, 1, d), (0, pitch, 0, 1), at)
        t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        return t
    for queries, keys in ((3, 200003), (150001, 40)):
        q, dy, k, v = far(queries, 0), far(queries, 128), far(keys, 256), far(keys, 512)
        lengths = _lengths(keys - 1)
        y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
        near = [t.contiguous() for t in (q, k, v)]
        y2, lse2 = ra.cross_attention(*near, key_lengths=lengths, stats=True)
        assert torch.equal(y, y2) and torch.equal(lse, lse2)
        for a, b in zip(ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths),
                        ra.cross_attention_backward(dy.contiguous(), *near, y, lse, key_lengths=lengths)):
            assert torch.equal(a, b)
        # the last rows, from the definition
        want, bound = L.attention(near[0][:, -3:], near[1], near[2], lengths)
        assert_within(y[:, -3:], want[0], bound[0], "y")


def test_many_sequences():
    """Each with its own number of keys; the fp64 form of the last ones."""
    b, n = 30011, 37
    print("case sequences", b, flush=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v, dy = (torch.randn(b, r, h, 64, device="cuda", generator=g).to(F16) for r, h in ((2, 4), (n, 2), (n, 2), (2, 4)))
    lengths = (torch.arange(b, device="cuda") % (n + 1)).int()
    y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
    grads = ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths)
    for part in (slice(0, 40), slice(b - 40, b)):
        args = [t[part] for t in (q, k, v)]
        want, bound = L.attention(*args, lengths[part])
        assert_within(y[part], want[0], bound[0], "y")
        want, bound = L.attention_backward(dy[part], *args, y[part], lse[part], lengths[part])
        for a, c, e, what in zip(grads, want, bound, ("dq", "dk", "dv")):
            assert_within(a[part], c, e, what)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_more_than_2_20_keys(dtype):
    """Values of 1: y is 1, whatever the weights; lse of like scores is their logarithm."""
    n = (1 << 20) + 77
    print("case keys", n, dtype, flush=True)
    q, k, v = torch.ones(1, 2, 4, 8, device="cuda"), torch.full((1, n, 2, 8), 0.25, device="cuda"), torch.ones(1, n, 2, 8, device="cuda")
    q, k, v = (t.to(dtype) for t in (q, k, v))
    y, lse = ra.cross_attention(q, k, v, scale=0.5, stats=True)
    # every weight is the same number, summed twice; sums of n terms in fp32
    assert ((y.double() - 1).abs() <= n * 2.0 ** -24 + torch.finfo(dtype).eps).all()
    assert ((lse.double() - (1 + torch.tensor(float(n)).double().log())).abs() <= n * 2.0 ** -24 + 1e-5).all()
    dy = torch.ones_like(q)
    dq, dk, dv = ra.cross_attention_backward(dy, q, k, v, y, lse, scale=0.5)
    # dv: the weights 1 / n of 2 queries and 2 heads; off by lse's own distance too
    off = 2 * n * 2.0 ** -24 + 1e-4 + torch.finfo(dtype).eps
    assert ((dv.double() * n / 4 - 1).abs() <= off + n * torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps).all()
    assert dq.isfinite().all() and dk.isfinite().all()
