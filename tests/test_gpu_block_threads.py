"""Block operators called by several host threads at once, each on its own
per-thread stream: every result is the one a single thread gets."""
import ctypes
import threading

import pytest
import torch

import ring_allreduce_reduce_amd as ra
from ring_allreduce_reduce_amd import block as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
PER_THREAD = 2                       # hipStreamPerThread


def _case(seed, rows, k, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s, scale=1.0: (torch.randn(*s, device="cuda", generator=g) * scale).to(BF16)  # noqa: E731
    x, w, dy, pre = rand(rows, k), rand(n, k, scale=k ** -0.5), rand(rows, n), rand(rows, n)
    return x, w, dy, pre


def _calls(x, w, dy, pre, outs, stream):
    """Forward (k split over blocks) and backward (dz, parts of sums, products)."""
    (rows, k), n = x.shape, w.shape[0]
    y, dx, dw, db = (t.data_ptr() for t in outs)
    fwd = B.ringar_linear_t(dtype=3, act=4, rows=rows, in_features=k, out_features=n, x=x.data_ptr(), ldx=k, weight=w.data_ptr(),
                            ldw=k, y=y, ldy=n)
    back = B.ringar_linear_backward_t(dtype=3, act=4, rows=rows, in_features=k, out_features=n, dy=dy.data_ptr(), lddy=n,
                                      pre=pre.data_ptr(), ldp=n, x=x.data_ptr(), ldx=k, weight=w.data_ptr(), ldw=k, dx=dx, lddx=k,
                                      dweight=dw, lddw=k, dbias=db)
    return (B._fn("ringar_linear")(ctypes.byref(fwd), stream), B._fn("ringar_linear_backward")(ctypes.byref(back), stream))


def test_threads_on_their_own_streams():
    print("case threads", flush=True)
    B._load()
    cases = [_case(i, rows, k, n) for i, (rows, k, n) in enumerate([(3, 8192, 256), (12, 4096, 520), (40, 4096, 256), (200, 1000, 520)])]
    outs = [[torch.full(s, float("nan"), dtype=BF16, device="cuda") for s in ((x.shape[0], w.shape[0]), x.shape, w.shape, (w.shape[0],))]
            for x, w, _, _ in cases]
    want = []
    for x, w, dy, pre in cases:
        want.append((ra.linear(x, w, act="silu"),) + ra.linear_backward(dy, x, w, pre, act="silu"))
    torch.cuda.synchronize()
    codes = []

    def work(i):
        for _ in range(25):
            codes.append(_calls(*cases[i], outs[i], PER_THREAD))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [(ra.SUCCESS, ra.SUCCESS)] * (25 * len(cases))
    for i, (a, b) in enumerate(zip(outs, want)):
        for got, ref, what in zip(a, b, ("y", "dx", "dweight", "dbias")):
            assert torch.equal(got, ref), (i, what)
