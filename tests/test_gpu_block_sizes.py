"""Products whose blocks are more than one launch takes: first, middle and
last outputs against the fp64 form, and zeros everywhere else."""
import pytest
import torch

import block_refs as R
import ring_allreduce_reduce_amd as ra

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gated", [False, True])
def test_more_columns_than_one_launch(gated, dtype):
    print("case columns", gated, dtype, flush=True)
    n = (1 << 26 if gated else 1 << 27) + 20
    at = [0, 15, 77777, (1 << 26) - 9, n - 21, n - 20, n - 1]
    x, some = _rand(1, 1, 8, dtype=dtype), _rand(2, 2 * len(at) if gated else len(at), 8, dtype=dtype)
    w = torch.zeros(2 * n if gated else n, 8, dtype=dtype, device="cuda")
    w[at] = some[:len(at)]
    if gated:
        w[[n + i for i in at]] = some[len(at):]
    y = (ra.gated_ffn if gated else ra.linear)(x, w, act="relu")
    want, bound = R.gated_forward(x, some, None, "relu") if gated else R.linear_forward(x, some, None, "relu", None)
    R.assert_within(y[:, at], want[0], bound[0], "y")
    assert int(torch.count_nonzero(y)) == int(torch.count_nonzero(y[:, at]))


def test_more_rows_than_one_launch():
    print("case rows", flush=True)
    rows = (1 << 30) + 100
    at = [0, 63, 1 << 20, (1 << 30) - 65, (1 << 30) - 1, 1 << 30, rows - 1]
    x = torch.zeros(rows, 8, dtype=BF16, device="cuda")
    x[at] = _rand(3, len(at), 8)
    w = _rand(4, 8, 8)
    y = ra.linear(x, w)
    want, bound = R.linear_forward(x[at], w, None, "none", None)
    R.assert_within(y[at], want[0], bound[0], "y")
    y[at] = 0
    assert not any(bool(part.any()) for part in y.split(1 << 27))
    dx, _, _ = ra.linear_backward(x, None, w, dweight=False, dbias=False)
    want, bound = R.backward(x[at], x[at], w, None, "none", False)
    R.assert_within(dx[at], want[0], bound[0], "dx")
    dx[at] = 0
    assert not any(bool(part.any()) for part in dx.split(1 << 27))
