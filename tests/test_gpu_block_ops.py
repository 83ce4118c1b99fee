"""Block operators on the GPU against their plain fp64 forms: types, sizes
from one token to long ones, odd widths, strides, alignments, empty inputs,
other streams, graph capture, and gradients against differences."""
import zlib

import pytest
import torch

import block_refs as R
import ring_allreduce_reduce_amd as ra

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [F32, F16, BF16]


def _gen(*key):
    print("case", *key, flush=True)
    g = torch.Generator()
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def _rand(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _inside(t, pad_rows=1, pad=5, shift=3, fill=float("nan")):
    """t as a view into a larger array of NaN: row stride and start that no
    alignment rule holds for."""
    big = torch.full((t.shape[0] + pad_rows, t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    v = big[:t.shape[0], shift:shift + t.shape[1]]
    v.copy_(t)
    return v


# ------------------------------------------------------------------ layer norm
NORM_SIZES = [(1, 1), (1, 64), (3, 7), (17, 128), (16, 129), (5, 512), (9, 513), (33, 1001), (4, 1024), (7, 2048), (3, 2049),
              (600, 40), (2, 4096), (5, 4100), (3, 8192), (2, 9001), (2, 16384), (2, 16385), (3, 40000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_layer_norm(rows, cols, dtype):
    g = _gen("norm", rows, cols, dtype)
    x = (_rand(g, (rows, cols), F32) + 0.5).to(dtype)
    w, b = _rand(g, (cols,), dtype), _rand(g, (cols,), dtype)
    got = ra.layer_norm(x, w, b, 1e-5, stats=True)
    want, bound = R.norm_forward(x, w, b, 1e-5)
    for a, c, e, what in zip(got, want, bound, ("y", "mean", "rstd")):
        R.assert_within(a, c, e, what)
    assert torch.equal(ra.layer_norm(x, w, b), got[0])
    dy = _rand(g, (rows, cols), dtype)
    grads = ra.layer_norm_backward(dy, x, got[1], got[2], w)
    want, bound = R.norm_backward(dy, x, got[1], got[2], w)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        R.assert_within(a, c, e, what)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("cols", [100, 3000, 20000])
def test_layer_norm_fp32_parameters(cols, dtype):
    g = _gen("norm fp32", cols, dtype)
    x, w, b = _rand(g, (11, cols), dtype), _rand(g, (cols,), F32), _rand(g, (cols,), F32)
    y, mean, rstd = ra.layer_norm(x, w, b, stats=True)
    want, bound = R.norm_forward(x, w, b, 1e-5)
    R.assert_within(y, want[0], bound[0], "y")
    dy = _rand(g, (11, cols), dtype)
    grads = ra.layer_norm_backward(dy, x, mean, rstd, w)
    assert grads[1].dtype == F32 and grads[2].dtype == F32
    want, bound = R.norm_backward(dy, x, mean, rstd, w)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        R.assert_within(a, c, e, what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [77, 1000, 2500, 17000])
def test_layer_norm_strided_without_parameters(cols, dtype):
    g = _gen("norm strided", cols, dtype)
    x = _inside(_rand(g, (6, cols), dtype))
    dy = _inside(_rand(g, (6, cols), dtype), pad=9, shift=1)
    big = torch.full((6, cols + 3), 7.0, dtype=dtype, device="cuda")
    y, mean, rstd = ra.layer_norm(x, stats=True, out=big[:, 2:2 + cols])
    want, bound = R.norm_forward(x, None, None, 1e-5)
    R.assert_within(y, want[0], bound[0], "y")
    assert (big[:, :2] == 7).all() and (big[:, 2 + cols:] == 7).all()
    grads = ra.layer_norm_backward(dy, x, mean, rstd)
    want, bound = R.norm_backward(dy, x, mean, rstd, None)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        R.assert_within(a, c, e, what)
    # each gradient alone is the same gradient
    assert torch.equal(ra.layer_norm_backward(dy, x, mean, rstd, dweight=False, dbias=False)[0], grads[0])
    assert torch.equal(ra.layer_norm_backward(dy, x, mean, rstd, dx=False, dbias=False)[1], grads[1])
    assert torch.equal(ra.layer_norm_backward(dy, x, mean, rstd, dx=False, dweight=False)[2], grads[2])


def test_layer_norm_in_place_constant_rows_and_nan_rows():
    for cols in (50, 700, 5000, 18000):
        _gen("norm special", cols)
        x = torch.randn(5, cols, generator=torch.Generator().manual_seed(cols)).cuda()
        x[1] = 3.25                     # variance zero
        x[2, cols // 2] = float("nan")
        x[3, 0] = float("inf")
        want = ra.layer_norm(x)
        assert (want[1] == 0).all() and want[2].isnan().all() and want[3].isnan().all()
        assert want[0].isfinite().all() and want[4].isfinite().all()
        y = x.clone()
        assert ra.layer_norm(y, out=y).data_ptr() == y.data_ptr()
        assert torch.equal(y[[0, 1, 4]], want[[0, 1, 4]])


def test_layer_norm_many_rows_and_dims():
    g = _gen("norm rows")
    x = _rand(g, (3, 1500, 96), BF16)
    w = _rand(g, (96,), BF16)
    y, mean, rstd = ra.layer_norm(x, w, stats=True)
    assert y.shape == x.shape and mean.shape == (3, 1500)
    want, bound = R.norm_forward(x, w, None, 1e-5)
    R.assert_within(y, want[0], bound[0], "y")
    dy = _rand(g, x.shape, BF16)
    grads = ra.layer_norm_backward(dy, x, mean, rstd, w)
    want, bound = R.norm_backward(dy, x, mean, rstd, w)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        R.assert_within(a, c, e, what)


# ------------------------------------------------------------------ products
# rows, in_features, out_features: single tokens, tiles' edges, odd widths
SIZES = [(1, 1, 1), (1, 64, 64), (1, 1000, 72), (2, 4096, 40), (5, 8, 300), (16, 520, 129), (17, 200, 256), (31, 1024, 16),
         (33, 7, 65), (64, 65, 31), (65, 128, 264), (100, 72, 1001), (127, 96, 128), (129, 264, 136), (200, 1003, 90),
         (256, 64, 256), (257, 192, 520), (300, 2056, 24), (513, 40, 24)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,n", SIZES)
@pytest.mark.parametrize("gated", [False, True])
def test_products(rows, k, n, dtype, gated):
    g = _gen("product", rows, k, n, dtype, gated)
    wide = 2 * n if gated else n
    act = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid", "none"][(rows + k + n) % 6]
    x, w = _rand(g, (rows, k), dtype), _rand(g, (wide, k), dtype, k ** -0.5)
    b = _rand(g, (wide,), dtype) if rows % 2 else None
    if gated:
        got = ra.gated_ffn(x, w, b, act=act, save_pre=True)
        want, bound = R.gated_forward(x, w, b, act)
    else:
        res = _rand(g, (rows, n), dtype) if n % 2 else None
        got = ra.linear(x, w, b, act=act, residual=res, save_pre=True)
        want, bound = R.linear_forward(x, w, b, act, res)
    for a, c, e, what in zip(got, want, bound, ("y", "pre")):
        R.assert_within(a, c, e, what)
    dy = _rand(g, (rows, n), dtype)
    back = ra.gated_ffn_backward if gated else ra.linear_backward
    grads = back(dy, x, w, got[1], act=act)
    want, bound = R.backward(dy, x, w, got[1], act, gated)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        R.assert_within(a, c, e, what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,k,n", [(3601, 3608, 3624), (5000, 72, 5016), (4200, 4160, 4136)])
def test_large_products(rows, k, n, gated, dtype):
    """The largest tiles, with edges and a ragged last step in every product."""
    g = torch.Generator(device="cuda")
    print("case large", rows, k, n, gated, dtype, flush=True)
    g.manual_seed(rows + k + n)
    rand = lambda *s, scale=1.0: (torch.randn(*s, device="cuda", generator=g) * scale).to(dtype)  # noqa: E731
    n = n // 2 if gated else n
    wide = 2 * n if gated else n
    x, w, b, dy = rand(rows, k), rand(wide, k, scale=k ** -0.5), rand(wide), rand(rows, n)
    res = None if gated else rand(rows, n)
    cuda64 = lambda *t: [None if v is None else _Cuda64(v) for v in t]  # noqa: E731
    if gated:
        got = ra.gated_ffn(x, w, b, act="silu", save_pre=True)
        want, bound = R.gated_forward(*cuda64(x, w, b), "silu")
    else:
        got = ra.linear(x, w, b, act="gelu_tanh", residual=res, save_pre=True)
        want, bound = R.linear_forward(*cuda64(x, w, b), "gelu_tanh", _Cuda64(res))
    for a, c, e, what in zip(got, want, bound, ("y", "pre")):
        _within_cuda(a, c, e, what)
    back = ra.gated_ffn_backward if gated else ra.linear_backward
    act = "silu" if gated else "gelu_tanh"
    grads = back(dy, x, w, got[1], act=act)
    want, bound = R.backward(*cuda64(dy, x, w, got[1]), act, gated)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        _within_cuda(a, c, e, what)


class _Cuda64:
    """A GPU tensor for the fp64 forms that stays on the GPU."""

    def __init__(self, t):
        self.t, self.dtype, self.shape = t, t.dtype, t.shape

    def double(self):
        return _Stay(self.t.double())


class _Stay:
    def __init__(self, t):
        self.t = t

    def cpu(self):
        return self.t


def _within_cuda(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), bad.nonzero()[:4].tolist(), float((off / bound).max()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,n", [(1, 520, 40), (20, 264, 72), (70, 135, 130), (300, 256, 264)])
@pytest.mark.parametrize("gated", [False, True])
def test_products_strided_in_nan(rows, k, n, dtype, gated):
    """Operands inside arrays of NaN, at odd strides: nothing outside is used."""
    g = _gen("strided", rows, k, n, dtype, gated)
    wide = 2 * n if gated else n
    for pad, shift in ((5, 3), (16, 8)):      # no row aligned; every row aligned
        x = _inside(_rand(g, (rows, k), dtype), pad=pad, shift=shift)
        w = _inside(_rand(g, (wide, k), dtype, k ** -0.5), pad=pad, shift=shift)
        dy = _inside(_rand(g, (rows, n), dtype), pad=pad, shift=shift)
        pre = _inside(_rand(g, (rows, wide), dtype), pad=pad, shift=shift)
        b = _rand(g, (wide,), dtype)
        big = torch.full((rows, n + pad), 7.0, dtype=dtype, device="cuda")
        out = big[:, shift:shift + n]
        if gated:
            ra.gated_ffn(x, w, b, act="silu", out=out)
            want, bound = R.gated_forward(x, w, b, "silu")
        else:
            res = _inside(_rand(g, (rows, n), dtype), pad=pad, shift=shift)
            ra.linear(x, w, b, act="silu", residual=res, out=out)
            want, bound = R.linear_forward(x, w, b, "silu", res)
        R.assert_within(out, want[0], bound[0], "y")
        assert (big[:, :shift] == 7).all() and (big[:, shift + n:] == 7).all()
        back = ra.gated_ffn_backward if gated else ra.linear_backward
        grads = back(dy, x, w, pre, act="silu")
        want, bound = R.backward(dy, x, w, pre, "silu", gated)
        for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
            R.assert_within(a, c, e, what)
        one = back(dy, x, w, pre, act="silu", dweight=False, dbias=False)
        assert torch.equal(one[0], grads[0]) and one[1] is None and one[2] is None
        one = back(dy, x, None, pre, act="silu", dx=False, dbias=False)
        assert torch.equal(one[1], grads[1]) and one[0] is None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,k,n", [(1, 1031, 1024), (2, 9, 120000), (3, 130000, 9), (4, 2056, 1030), (5, 1024, 1100), (8, 100, 10490),
                                      (9, 1040, 1040)])
def test_few_rows_backward(rows, k, n, gated, dtype):
    """The gradients of a few rows through a weight of a million values."""
    g = _gen("few", rows, k, n, gated, dtype)
    wide = 2 * n if gated else n
    act = "gelu" if rows % 2 else "silu"
    back = ra.gated_ffn_backward if gated else ra.linear_backward
    dy, x, w, pre = _rand(g, (rows, n), dtype), _rand(g, (rows, k), dtype), _rand(g, (wide, k), dtype, wide ** -0.5), _rand(g, (rows, wide), dtype)
    for place in (lambda t: t, lambda t: _inside(t, pad=5, shift=3)):
        dy1, x1, w1, pre1 = place(dy), place(x), place(w), place(pre)
        grads = back(dy1, x1, w1, pre1, act=act)
        want, bound = R.backward(dy, x, w, pre, act, gated)
        for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
            R.assert_within(a, c, e, what)
        for which in range(3):
            names = ("dx", "dweight", "dbias")
            one = back(dy1, x1, w1, pre1, act=act, **{v: False for v in names if v != names[which]})
            assert sum(v is not None for v in one) == 1
            R.assert_within(one[which], want[which], bound[which], names[which] + " alone")
    if not gated:
        grads = back(dy, x, w)                      # no activation
        want, bound = R.backward(dy, x, w, None, "none", False)
        for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
            R.assert_within(a, c, e, what)


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_broadcast_rows_and_residual_in_place(dtype):
    g = _gen("broadcast", dtype)
    x1, w, r1 = _rand(g, (1, 136), dtype), _rand(g, (72, 136), dtype, 0.1), _rand(g, (1, 72), dtype)
    x, r = x1.expand(50, 136), r1.expand(50, 72)
    want, bound = R.linear_forward(x, w, None, "none", r)
    R.assert_within(ra.linear(x, w, residual=r), want[0], bound[0], "y")
    y = r.contiguous()
    assert ra.linear(x, w, residual=y, out=y).data_ptr() == y.data_ptr()
    R.assert_within(y, want[0], bound[0], "y in place")
    dy = _rand(g, (1, 72), dtype).expand(50, 72)
    grads = ra.linear_backward(dy, x, w)
    want, bound = R.backward(dy, x, w, None, "none", False)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        R.assert_within(a, c, e, what)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
def test_activations_over_their_range(act, dtype):
    """Pre-activations from far negative to far positive, each act and slope."""
    _gen("acts", act, dtype)
    z = torch.linspace(-30, 30, 481).to(dtype).cuda().reshape(1, -1)
    one = torch.ones(1, 1, dtype=dtype, device="cuda")
    y = ra.linear(one, z.T.contiguous(), act=act)
    want, bound = R.linear_forward(one, z.T, None, act, None)
    R.assert_within(y, want[0], bound[0], "act")
    dy = torch.ones_like(z)
    if act != "none":
        got = ra.linear_backward(dy, one, z.T.contiguous(), z, act=act)
        want, bound = R.backward(dy, one, z.T, z, act, False)
        for a, c, e, what in zip(got, want, bound, ("dx", "dweight", "dbias")):
            R.assert_within(a, c, e, what)
    # the far ends, infinities and NaN
    ends = torch.tensor([[-3e4, 3e4, float("inf"), float("nan")]], device="cuda").to(dtype)
    y = ra.linear(one, ends.T.contiguous(), act=act).float().cpu().flatten()
    plain = R.act64(act, ends.double().cpu().flatten())
    assert torch.equal(y[:2], plain[:2].to(dtype).float()) or act == "none"
    assert y[2] == (1.0 if act == "sigmoid" else float("inf")) and y[3].isnan()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [3, 70, 300])
def test_nan_and_inf_stay_in_their_row_and_column(rows, dtype):
    g = _gen("nan rows", rows, dtype)
    x, w = _rand(g, (rows, 72), dtype), _rand(g, (80, 72), dtype)
    clean = ra.linear(x, w)
    x[1, 5], w[7, 3] = float("nan"), float("inf")
    y = ra.linear(x, w)
    keep_r = [r for r in range(rows) if r != 1]
    keep_c = [c for c in range(80) if c != 7]
    assert y[1].isnan().all() and not y[keep_r][:, 7].isfinite().any()
    assert torch.equal(y[keep_r][:, keep_c], clean[keep_r][:, keep_c])


@pytest.mark.parametrize("dtype", TYPES)
def test_nothing_to_do(dtype):
    _gen("empty", dtype)
    e = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    w = torch.ones(24, 16, dtype=dtype, device="cuda")
    assert ra.linear(e(0, 16), w).shape == (0, 24)
    assert ra.gated_ffn(e(2, 0, 16), w).shape == (2, 0, 12)
    assert ra.layer_norm(e(0, 16)).shape == (0, 16)
    dx, dw, db = ra.linear_backward(e(0, 24), e(0, 16), w, e(0, 24), act="silu")
    assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()
    dx, dw, db = ra.gated_ffn_backward(e(0, 12), e(0, 16), w, e(0, 24))
    assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()
    stats = torch.empty(0, device="cuda")
    dx, dw, db = ra.layer_norm_backward(e(0, 16), e(0, 16), stats, stats)
    assert (dw == 0).all() and (db == 0).all()
    # no inner features: the sum is empty
    y = ra.linear(e(3, 0), e(5, 0), torch.full((5,), 2.0, dtype=dtype, device="cuda"), act="relu")
    assert (y == 2).all()
    dx, dw, db = ra.linear_backward(torch.ones(3, 5, dtype=dtype, device="cuda"), e(3, 0), e(5, 0))
    assert dx.shape == (3, 0) and dw.shape == (5, 0) and (db == 3).all()
    # no outputs: x's gradient is zero
    dx, dw, db = ra.linear_backward(e(3, 0), torch.ones(3, 16, dtype=dtype, device="cuda"), e(0, 16))
    assert (dx == 0).all() and dw.shape == (0, 16) and db.shape == (0,)


@pytest.mark.parametrize("gated", [False, True])
def test_long_sums_and_split_k(gated):
    """Few outputs, a long inner dimension: k is split and joined in order, so
    results repeat bit for bit."""
    for dtype, k in ((BF16, 30000), (F16, 16392), (F32, 20001)):
        g = _gen("long", dtype, k, gated)
        x, w = _rand(g, (40, k), dtype), _rand(g, (48, k), dtype, k ** -0.5)
        f = ra.gated_ffn if gated else ra.linear
        y = f(x, w, act="gelu")
        want, bound = (R.gated_forward(x, w, None, "gelu") if gated else R.linear_forward(x, w, None, "gelu", None))
        R.assert_within(y, want[0], bound[0], "y")
        for _ in range(3):
            assert torch.equal(f(x, w, act="gelu"), y)
        n = 24 if gated else 48
        rows = k // 4
        dy, x2, pre = _rand(g, (rows, n), dtype), _rand(g, (rows, 64), dtype), _rand(g, (rows, 48), dtype)
        w2 = _rand(g, (48, 64), dtype)
        back = ra.gated_ffn_backward if gated else ra.linear_backward
        grads = back(dy, x2, w2, pre, act="silu")
        want, bound = R.backward(dy, x2, w2, pre, "silu", gated)
        for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
            R.assert_within(a, c, e, what)
        for a, b in zip(back(dy, x2, w2, pre, act="silu"), grads):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """A row stride that puts the last rows past 2^32 bytes (and 2^31 elements)."""
    _gen("far rows")
    rows, k = 2, 64
    ld = (1 << 31) - 8
    big = torch.zeros(ld + k, dtype=BF16, device="cuda")
    x = torch.as_strided(big, (rows, k), (ld, 1))
    g = torch.Generator().manual_seed(5)
    x.copy_(_rand(g, (rows, k), BF16))
    w = _rand(g, (32, k), BF16)
    want, bound = R.linear_forward(x, w, None, "none", None)
    R.assert_within(ra.linear(x, w), want[0], bound[0], "y")
    y, mean, rstd = ra.layer_norm(x, stats=True)
    want, bound = R.norm_forward(x, None, None, 1e-5)
    R.assert_within(y, want[0], bound[0], "norm")
    dy = _rand(g, (rows, 32), BF16)
    grads = ra.linear_backward(dy, x, w)
    want, bound = R.backward(dy, x, w, None, "none", False)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        R.assert_within(a, c, e, what)


def test_many_rows_beyond_32_bit_offsets():
    """rows * in_features past 2^31 elements: first, middle and last rows."""
    _gen("tall")
    rows, k, n = (1 << 31) // 1024 + 300, 1024, 8
    x = torch.zeros(rows, k, dtype=BF16, device="cuda")
    at = [0, 1, 1 << 20, (1 << 21) - 1, 1 << 21, rows - 1]
    g = torch.Generator().manual_seed(9)
    x[at] = _rand(g, (len(at), k), BF16)
    w, b = _rand(g, (n, k), BF16), _rand(g, (n,), BF16)
    y = ra.linear(x, w, b)
    want, bound = R.linear_forward(x[at], w, b, "none", None)
    R.assert_within(y[at], want[0], bound[0], "y")
    mask = torch.ones(rows, dtype=torch.bool, device="cuda")
    mask[at] = False
    assert torch.equal(y[mask][::4097].unique(dim=0), b[None])
    h = ra.layer_norm(x, b.new_ones(k))
    want, bound = R.norm_forward(x[at], None, None, 1e-5)
    R.assert_within(h[at], want[0], bound[0], "norm")


# ------------------------------------------------------------------ streams
def test_other_stream_and_first_use():
    g = _gen("stream")
    st = torch.cuda.Stream()
    x, w = _rand(g, (130, 264), BF16), _rand(g, (520, 264), BF16, 0.06)
    b = _rand(g, (520,), BF16)
    want, pre = ra.gated_ffn(x, w, b, save_pre=True)
    dy = _rand(g, (130, 260), BF16)
    grads = ra.gated_ffn_backward(dy, x, w, pre)
    torch.cuda.synchronize()
    for _ in range(3):
        y, p = ra.gated_ffn(x, w, b, save_pre=True, stream=st)
        back = ra.gated_ffn_backward(dy, x, w, p, stream=st)
        n = ra.layer_norm(y, stream=st)
        st.synchronize()
        assert torch.equal(y, want) and all(torch.equal(a, c) for a, c in zip(back, grads))
        assert torch.equal(n, ra.layer_norm(want))
    ra.ringar_release()
    assert all(torch.equal(a, c) for a, c in zip(ra.gated_ffn_backward(dy, x, w, pre), grads))


def test_capture_and_replay():
    """A block's forward and backward pass in a graph, replayed on new inputs
    with eager work between the replays."""
    g = _gen("capture")
    x, w, wd = _rand(g, (50, 264), BF16), _rand(g, (272, 264), BF16, 0.06), _rand(g, (264, 136), BF16, 0.08)
    nw, nb, dy = _rand(g, (264,), BF16), _rand(g, (264,), BF16), _rand(g, (50, 264), BF16)

    def step():
        n, mean, rstd = ra.layer_norm(x, nw, nb, stats=True)
        h, pre = ra.gated_ffn(n, w, save_pre=True)
        y = ra.linear(h, wd, residual=x)
        dh, dwd, _ = ra.linear_backward(dy, h, wd, dbias=False)
        dn, dw, db = ra.gated_ffn_backward(dh, n, w, pre)
        return (y, dwd, dw, db) + ra.layer_norm_backward(dn, x, mean, rstd, nw)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        outs = step()
    for i in range(4):
        x.copy_(_rand(g, x.shape, BF16))
        dy.copy_(_rand(g, dy.shape, BF16))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, c) in enumerate(zip(outs, want)):
            assert torch.equal(a, c), (i, k)


def test_capture_without_a_workspace_is_refused():
    _gen("capture refused")
    st = torch.cuda.Stream()
    x, w, dy = (torch.ones(s, dtype=BF16, device="cuda") for s in ((64, 64), (64, 64), (64, 64)))
    graph = torch.cuda.CUDAGraph()
    ra.ringar_release()
    with torch.cuda.graph(graph, stream=st):
        with pytest.raises(ra.RingarError) as e:
            ra.linear_backward(dy, x, w, dy, act="silu")
        y = ra.layer_norm(x)
    assert e.value.code == ra.INVALID_USAGE and "capture" in str(e.value)
    graph.replay()
    torch.cuda.synchronize()
    assert (y == 0).all()


# ------------------------------------------------------------------ gradients against differences
def _loss(outs, dy):
    return float((outs.double().cpu() * dy.double().cpu()).sum())


@pytest.mark.parametrize("op", ["layer_norm", "linear", "gated_ffn"])
def test_gradients_against_differences(op):
    """Central differences of the fp32 forward pass along random directions.
    Allowed: what the plain fp64 form's own difference is off by, the forward
    bounds over the step, and the gradients' bounds along the direction."""
    g = _gen("differences", op)
    rows, k, n, h = 20, 40, 24, 2.0 ** -6
    x, dy = _rand(g, (rows, k), F32), _rand(g, (rows, k if op == "layer_norm" else n), F32)
    if op == "layer_norm":
        w, b = _rand(g, (k,), F32), _rand(g, (k,), F32)
        run = lambda x, w, b: ra.layer_norm(x, w, b)  # noqa: E731
        ref = lambda x, w, b: R.norm_forward(x, w, b, 1e-5)  # noqa: E731
        _, mean, rstd = ra.layer_norm(x, w, b, stats=True)
        grads = ra.layer_norm_backward(dy, x, mean, rstd, w)
        want, bound = R.norm_backward(dy, x, mean, rstd, w)
    else:
        gated = op == "gated_ffn"
        w, b = _rand(g, (2 * n if gated else n, k), F32, 0.2), _rand(g, (2 * n if gated else n,), F32)
        f = getattr(ra, op)
        run = lambda x, w, b: f(x, w, b, act="gelu")  # noqa: E731
        ref = ((lambda x, w, b: R.gated_forward(x, w, b, "gelu")) if gated
               else (lambda x, w, b: R.linear_forward(x, w, b, "gelu", None)))
        _, pre = f(x, w, b, act="gelu", save_pre=True)
        grads = getattr(ra, op + "_backward")(dy, x, w, pre, act="gelu")
        want, bound = R.backward(dy, x, w, pre, "gelu", gated)
    for i in range(3):
        args = [x, w, b]
        d = _rand(g, args[i].shape, F32)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        step = (up[i].double() - down[i].double()).cpu()              # as rounded
        got = _loss(run(*up), dy) - _loss(run(*down), dy)
        (u64, ub), (d64, db) = ref(*up), ref(*down)
        plain = _loss(u64[0], dy) - _loss(d64[0], dy)
        noise = float(((ub[0] + db[0]) * dy.double().cpu().abs()).sum())
        along = float((grads[i].double().cpu().reshape(step.shape) * step).sum())
        along64 = float((want[i].reshape(step.shape) * step).sum())
        slack = float((bound[i].reshape(step.shape) * step.abs()).sum())
        # pre and the statistics are fp32 roundings of the pass's own: their effect is within twice the bounds
        assert abs(got - along) <= abs(plain - along64) + noise + 2 * slack, (op, i, got, along, plain, along64)


def test_flags_must_be_flags():
    x, w = torch.ones(2, 8, device="cuda"), torch.ones(4, 8, device="cuda")
    for call in (lambda: ra.linear_backward(torch.ones(2, 4, device="cuda"), x, w, dx=x), lambda: ra.layer_norm(x, stats=x),
                 lambda: ra.linear(x, w, save_pre=1)):
        with pytest.raises(ra.RingarError, match="must be True or False"):
            call()


@pytest.mark.parametrize("rows", [1, 3, 12, 20])
def test_weight_beyond_32_bit_offsets(rows):
    """out_features * in_features past 2^31 elements, forward and backward:
    first, middle and last rows of the weight."""
    k, n = 2048, (1 << 31) // 2048 + 300
    g = _gen("wide", rows)
    at = [0, 1, 77777, (1 << 20) - 1, 1 << 20, n - 1]
    x, some = _rand(g, (rows, k), BF16), _rand(g, (len(at), k), BF16, k ** -0.5)
    w = torch.zeros(n, k, dtype=BF16, device="cuda")
    w[at] = some
    y = ra.linear(x, w)
    want, bound = R.linear_forward(x, some, None, "none", None)
    R.assert_within(y[:, at], want[0], bound[0], "y")
    assert int(torch.count_nonzero(y)) == int(torch.count_nonzero(y[:, at]))
    dy = torch.zeros(rows, n, dtype=BF16, device="cuda")
    dy[:, at] = _rand(g, (rows, len(at)), BF16)
    del y
    dx, dw, db = ra.linear_backward(dy, x, w)
    want, bound = R.backward(dy[:, at].contiguous(), x, some, None, "none", False)
    R.assert_within(dx, want[0], bound[0], "dx")
    R.assert_within(dw[at], want[1], bound[1], "dweight")
    R.assert_within(db[at], want[2], bound[2], "dbias")
    dw[at] = 0
    assert int(torch.count_nonzero(dw.view(-1, 1 << 11)[::1009])) == 0 and int(torch.count_nonzero(dw[-400:])) == 0
