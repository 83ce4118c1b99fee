"""Two host threads in attention, norm and dropout at once, started together: the
results of every iteration, not of the last one alone, are those of the calls alone."""
import threading

import pytest
import torch

from test_gpu_layer_threads import operands, work

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", [False, True])
def test_every_iteration(shared):
    sets = [operands(seed) for seed in (1, 2)]
    alone = [work(ops) for ops in sets]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    streams = [one, one if shared else torch.cuda.Stream()]
    got, errors, together = [[], []], [], threading.Barrier(2)

    def run(i):
        try:
            work(sets[i], streams[i])          # the first call's allocations
            together.wait(timeout=60)
            for _ in range(20):
                got[i].append(work(sets[i], streams[i]))
        except Exception as e:
            together.abort()
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for want, runs in zip(alone, got):
        assert len(runs) == 20
        for n, results in enumerate(runs):
            for i, (x, y) in enumerate(zip(want, results)):
                assert torch.equal(x, y), (n, i)
