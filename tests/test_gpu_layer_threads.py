"""Two host threads in attention, norm and dropout at once, each on a stream of
its own and both on one: the results are those of the calls alone, bit for bit."""
import threading

import pytest
import torch

import ring_allreduce_reduce_amd as ra

pytestmark = pytest.mark.gpu


def operands(seed):
    g = torch.Generator().manual_seed(seed)
    make = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    return make(2, 3, 8, 64), make(2, 1500 + 100 * seed, 4, 64), make(2, 1500 + 100 * seed, 4, 64), make(37, 1000), make(1000)


def work(ops, stream=None):
    q, k, v, x, w = ops
    y, lse = ra.cross_attention(q, k, v, stats=True, stream=stream)                 # keys in parts: a workspace
    grads = ra.cross_attention_backward(y, q, k, v, y, lse, stream=stream)
    n, s, rstd = ra.rms_norm(x, w, residual=x, stats=True, stream=stream)
    norm = ra.rms_norm_backward(n, s, rstd, w, stream=stream)                       # partial rows: the same one
    return [y, lse, *grads, n, s, rstd, *norm, ra.dropout(x, 0.3, 5, 7, residual=n, stream=stream)]


@pytest.mark.parametrize("shared", [False, True])
def test_two_threads(shared):
    sets = [operands(seed) for seed in (1, 2)]
    alone = [work(ops) for ops in sets]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    streams = [one, one if shared else torch.cuda.Stream()]
    got, errors = [None, None], []

    def run(i):
        try:
            for _ in range(20):
                got[i] = work(sets[i], streams[i])
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
