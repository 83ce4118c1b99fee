"""How near the block operators come to their fp64 forms where a bound on
single values leaves room: values that are rounded once, and norms."""
import zlib

import pytest
import torch

import block_refs as R
import ring_allreduce_reduce_amd as ra

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _gen(*key):
    print("case", *key, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return lambda *s, dtype=F32, scale=1.0: (torch.randn(*s, device="cuda", generator=g) * scale).to(dtype)


def _dz64(dy, pre, act, gated):
    """dz in fp64, and what evaluating it in fp32 may be off by."""
    dt = dy.dtype
    dy, pre = dy.double().cpu(), pre.double().cpu()
    n = dy.shape[1]
    if gated:
        g, u = pre[:, :n], pre[:, n:]
        dz = torch.cat((dy * u * R.act64_grad(act, g), dy * R.act64(act, g)), 1)
        e = torch.cat(((dy * u).abs(), dy.abs()), 1) * R.act_error(dt, torch.cat((g, g), 1))
    else:
        dz = dy * R.act64_grad(act, pre)
        e = dy.abs() * R.act_error(dt, pre)
    return dz, e + 4 * R.U32 * dz.abs()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,k,n", [(1, 1031, 1024), (2, 64, 72), (3, 264, 1100), (4, 2056, 130)])
def test_gradients_of_few_rows_are_rounded_once(rows, k, n, gated, dtype):
    """dz of a few rows stays in fp32: dx and dweight carry one rounding to
    their type beside the fp32 sums'."""
    rand = _gen("few once", rows, k, n, gated, dtype)
    wide = 2 * n if gated else n
    dy, x, w, pre = rand(rows, n, dtype=dtype), rand(rows, k, dtype=dtype), rand(wide, k, dtype=dtype), rand(rows, wide, dtype=dtype)
    back = ra.gated_ffn_backward if gated else ra.linear_backward
    dx, dw, _ = back(dy, x, w, pre, act="silu")
    dz, e = _dz64(dy, pre, "silu", gated)
    x, w = x.double().cpu(), w.double().cpu()
    want = dz @ w
    R.assert_within(dx, want, R.rounded(dtype, want, e @ w.abs() + R.mm_error(dz.abs() + e, w, wide)), "dx")
    want = dz.T @ x
    R.assert_within(dw, want, R.rounded(dtype, want, e.T @ x.abs() + R.mm_error((dz.abs() + e).T, x, rows)), "dweight")
