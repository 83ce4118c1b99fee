"""Attention on rows that lie over each other (one row for all keys or queries, or
windows of one run of values): what lies where the next row would be belongs to the
rows before, infinities too.  The results are those on copies of the rows, bit for
bit."""
import pytest
import torch

import ring_allreduce_reduce_amd as ra
from attention_forms import CASES, F32, lengths_of

pytestmark = pytest.mark.gpu
INF = float("inf")


def _same(a, b, what):
    torch.testing.assert_close(a, b, rtol=0, atol=0, equal_nan=True, msg=lambda m: f"{what}: {m}")


def _rows(g, dtype, b, n, h, d, apart):
    """(b, n, h, d) whose rows are `apart` values from each other."""
    run = torch.randn(b, h, (n - 1) * apart + d, device="cuda", generator=g).to(dtype)
    # the last value of all is infinite: of the last row's last column, and of every row's where they are one
    run[:, :, -1] = INF
    return run.as_strided((b, n, h, d), (run.stride(0), apart, run.stride(1), 1))


def _check(dtype, b, lq, n, h, kv, d, lengths):
    print("case", dtype, b, lq, n, h, kv, d, flush=True)
    g = torch.Generator(device="cuda").manual_seed(n + d)
    each = 16 // dtype.itemsize
    lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q, k = (torch.randn(b, r, c, d, device="cuda", generator=g).to(dtype) for r, c in ((lq, h), (n, kv)))
    for apart in (0, each):
        if apart and (d * dtype.itemsize) % 16:
            continue
        v = _rows(g, dtype, b, n, kv, d - d % each, apart)
        y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
        want, _ = ra.cross_attention(q, k, v.contiguous(), key_lengths=lengths, stats=True)
        _same(y, want, ("y", apart))
        assert torch.isinf(y[0, :, :, -1]).all()
        dy = _rows(g, dtype, b, lq, h, d, apart)
        y = torch.randn(q.shape, device="cuda", generator=g).to(dtype)
        for name, a, c in zip(("dq", "dk", "dv"), ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths),
                              ra.cross_attention_backward(dy.contiguous(), q, k, v.contiguous(), y, lse, key_lengths=lengths)):
            _same(a, c, (name, apart))
        assert torch.isinf(c[0, :, :, -1]).all()


@pytest.mark.parametrize("dtype", [F32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,lq,n,h,kv,d", [(2, 1, 700, 4, 2, 64), (2, 37, 70, 4, 2, 128), (2, 3, 33, 2, 1, 40), (3, 65, 300, 2, 2, 96)])
def test_few_rows(b, lq, n, h, kv, d, dtype):
    _check(dtype, b, lq, n, h, kv, d, [n - 7 * i for i in range(b)])


@pytest.mark.parametrize("dtype,waves,parts,b,lq,n,h,kv,d", CASES)
def test_many_rows(dtype, waves, parts, b, lq, n, h, kv, d):
    _check(dtype, b, lq, n, h, kv, d, lengths_of(dtype, n))
