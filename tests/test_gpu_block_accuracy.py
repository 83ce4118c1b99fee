"""How near the block operators come to their fp64 forms where a bound on
single values leaves room: values that are rounded once, and norms."""
import zlib

import pytest
import torch

import block_refs as R
from block_norms import ONE_ROUNDING, TWO_ROUNDINGS, distance
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


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,k,n", [(3600, 3608, 3624), (5000, 72, 5016), (7500, 64, 48), (40, 20008, 48), (333, 1023, 2050), (16, 8192, 520)])
def test_products_sum_in_fp32(rows, k, n, gated, dtype):
    """Relative distances of whole outputs (test_block_bounds_cpu.py: what the
    bounds come from, and that sums in the type miss them)."""
    rand = _gen("norms", rows, k, n, gated, dtype)
    n = n // 2 if gated else n
    wide = 2 * n if gated else n
    x, w, dy = rand(rows, k, dtype=dtype), rand(wide, k, dtype=dtype, scale=k ** -0.5), rand(rows, n, dtype=dtype)
    y, pre = (ra.gated_ffn if gated else ra.linear)(x, w, act="silu", save_pre=True)
    z = x.double() @ w.double().T
    act = R.act64("silu", z[:, :n]) * z[:, n:] if gated else R.act64("silu", z)
    assert distance(pre, z) <= ONE_ROUNDING * R.UNIT[dtype]
    assert distance(y, act) <= ONE_ROUNDING * R.UNIT[dtype]
    dx, dw, _ = (ra.gated_ffn_backward if gated else ra.linear_backward)(dy, x, w, pre, act="silu")
    pre, dy = pre.double(), dy.double()
    slope = R.act64_grad("silu", pre[:, :n])
    dz = torch.cat((dy * pre[:, n:] * slope, dy * R.act64("silu", pre[:, :n])), 1) if gated else dy * slope
    assert distance(dx, dz @ w.double()) <= TWO_ROUNDINGS * R.UNIT[dtype]
    assert distance(dw, dz.T @ x.double()) <= TWO_ROUNDINGS * R.UNIT[dtype]


def _gelu_error(dtype, z):
    """Relative: the 16-bit types' polynomial (2.2e-5 beyond |z| = 4), the
    exponential's and erfc's argument, rounded to fp32 (a relative u32 of it is
    z^2 u32 of them), and a few operations."""
    poly = 2.0 ** -15 if dtype != F32 else 0.0
    return poly + (8 + 4 * z * z) * R.U32


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_gelu_in_its_lower_tail(dtype):
    """Values and slopes relative to themselves, down to z = -12, where the
    distribution is 1e-33."""
    _gen("gelu tail", dtype)
    z = torch.cat((torch.linspace(-12, 12, 961), torch.linspace(-1, 1, 801))).to(dtype).cuda().reshape(1, -1)
    z64 = z.double().cpu()
    # erfc: torch.special.ndtr cancels, to nothing at -8.3
    cdf, density = 0.5 * torch.special.erfc(-z64 * 0.5 ** 0.5), torch.exp(-z64 * z64 / 2) / (2 * torch.pi) ** 0.5
    err = _gelu_error(dtype, z64)
    y = ra.linear(torch.ones(1, 1, dtype=dtype, device="cuda"), z.T.contiguous(), act="gelu")
    want = z64 * cdf
    R.assert_within(y, want, R.rounded(dtype, want, err * want.abs()), "gelu")
    _, _, slope = ra.linear_backward(torch.ones_like(z), None, None, z, act="gelu", dx=False, dweight=False)
    want = cdf + z64 * density
    R.assert_within(slope, want[0], R.rounded(dtype, want, err * (cdf + (z64 * density).abs()))[0], "slope")


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slopes_where_the_square_overflows(act, dtype):
    """Finite pre-activations far out: the slope is its limit, 0 or 1."""
    _gen("far slopes", act, dtype)
    z = torch.tensor([[2e18, 2e19, 1e25, 3e38]], device="cuda").to(dtype)
    for sign, limit in ((1, 0.0 if act == "sigmoid" else 1.0), (-1, 0.0)):
        _, _, slope = ra.linear_backward(torch.ones_like(z), None, None, sign * z, act=act, dx=False, dweight=False)
        assert (slope == limit).all(), (sign, slope)
        # the gated form, as the products of few rows take it
        _, _, both = ra.gated_ffn_backward(torch.ones_like(z), None, None, torch.cat((sign * z, torch.ones_like(z)), 1), act=act, dx=False,
                                           dweight=False)
        assert (both[:4] == limit).all(), (sign, both)
    nan = torch.full_like(z, float("nan"))
    if act != "relu":
        assert ra.linear_backward(torch.ones_like(z), None, None, nan, act=act, dx=False, dweight=False)[2].isnan().all()
