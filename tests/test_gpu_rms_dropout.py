"""The root-mean-square norm and dropout on the GPU against their plain fp64
forms: types, sizes from one token to long rows, odd widths, strides, 8-bit
outputs, in place, captured calls, and gradients."""
import zlib

import numpy as np
import pytest
import torch

import layer_refs as L
import ring_allreduce_reduce_amd as ra
from block_refs import TINY, U32, UNIT, assert_within, rounded

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [F32, F16, BF16]
NAN, INF = float("nan"), float("inf")


def _gen(*key):
    print("case", *key, flush=True)
    g = torch.Generator()
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def _rand(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _inside(t, pad=5, shift=3):
    """t as a view into a larger array of NaN, at no alignment."""
    big = torch.full((t.shape[0] + 1, t.shape[1] + pad), NAN, dtype=t.dtype, device=t.device)
    v = big[:t.shape[0], shift:shift + t.shape[1]]
    v.copy_(t)
    return v


def _sum(x, r):
    """x + r as the kernel rounds it: the fp32 sum, rounded once."""
    return (x.float() + r.float()).to(x.dtype)


ROWS = [(1, 1), (1, 64), (3, 7), (17, 128), (16, 129), (5, 512), (9, 513), (33, 1001), (4, 1024), (7, 2048), (3, 2049), (600, 40),
        (2, 4096), (5, 4100), (3, 8192), (2, 9001), (2, 16384), (2, 16385), (3, 40000)]


def _check_fp8(q, scale, s, w, eps, group, what):
    """Scales within the norm's error; every byte within one rounding of its value."""
    (y, _), (ey, _) = L.rms_forward(s, w, eps)
    cols = y.shape[1]
    wide = group or cols
    n = -(-cols // wide)
    assert scale.shape[-1] == n and scale.dtype == F32 and q.dtype == torch.float8_e4m3fn
    scale = scale.double().cpu().reshape(-1, n)
    pad = lambda t: torch.nn.functional.pad(t, (0, n * wide - cols)).reshape(-1, n, wide)  # noqa: E731
    want = (pad(y).abs().amax(-1) / L.LARGEST).clamp(min=2.0 ** -126)
    off = pad(ey).amax(-1) / L.LARGEST + 2 * U32 * want
    assert ((scale - want).abs() <= off).all(), what
    each = scale.repeat_interleave(wide, 1)[:, :cols]
    z, ez = y / each, ey / each + 4 * U32 * (y / each).abs()
    got = q.float().double().cpu().reshape(z.shape)
    # 4 significant bits: half a step is 2^-4 of the value, of those below 2^-6 half their spacing of 2^-9
    bound = ez + torch.maximum(2.0 ** -4 * (z.abs() + ez), torch.tensor(2.0 ** -10).double())
    assert_within(got, z, bound, what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", ROWS)
def test_rms_norm(rows, cols, dtype):
    g = _gen("rms", rows, cols, dtype)
    x, r = _rand(g, (rows, cols), dtype, 2.0), _rand(g, (rows, cols), dtype)
    w = _rand(g, (cols,), dtype)
    y, s, rstd = ra.rms_norm(x, w, 1e-5, residual=r, stats=True)
    assert torch.equal(s, _sum(x, r))
    (want, er), (ey, ee) = L.rms_forward(s, w, 1e-5)
    assert_within(y, want, rounded(dtype, want, ey), "y")
    assert_within(rstd, er, ee, "rstd")
    assert torch.equal(ra.rms_norm(s, w, 1e-5), y)
    assert torch.equal(ra.rms_norm(x, w, 1e-5, residual=r)[0], y)
    for group in (None, 128):
        q, scale, s8, rstd8 = ra.rms_norm_fp8(x, w, 1e-5, residual=r, group=group, stats=True)
        assert torch.equal(s8, s) and torch.equal(rstd8, rstd) and q.shape == x.shape
        _check_fp8(q, scale, s, w, 1e-5, group, ("fp8", group))
        q2, scale2 = ra.rms_norm_fp8(s, w, 1e-5, group=group)
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(scale2, scale)
    dy, ds = _rand(g, (rows, cols), dtype), _rand(g, (rows, cols), dtype)
    for dsum in (ds, None):
        grads = ra.rms_norm_backward(dy, s, rstd, w, dsum=dsum)
        want, bound = L.rms_backward(dy, s, rstd, w, dsum)
        for a, c, e, what in zip(grads, want, bound, ("dx", "dweight")):
            assert_within(a, c, e, what)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("cols", [100, 3000, 20000])
def test_rms_norm_fp32_weight(cols, dtype):
    g = _gen("rms fp32", cols, dtype)
    x, w = _rand(g, (11, cols), dtype), _rand(g, (cols,), F32)
    y, rstd = ra.rms_norm(x, w, stats=True)
    (want, _), (ey, _) = L.rms_forward(x, w, 1e-6)
    assert_within(y, want, rounded(dtype, want, ey), "y")
    _check_fp8(*ra.rms_norm_fp8(x, w, group=128), x, w, 1e-6, 128, "fp8")
    dy = _rand(g, (11, cols), dtype)
    grads = ra.rms_norm_backward(dy, x, rstd, w)
    assert grads[1].dtype == F32
    want, bound = L.rms_backward(dy, x, rstd, w, None)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight")):
        assert_within(a, c, e, what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [77, 1000, 2500, 17000])
def test_rms_norm_strided(cols, dtype):
    g = _gen("rms strided", cols, dtype)
    x, r = _inside(_rand(g, (6, cols), dtype)), _inside(_rand(g, (6, cols), dtype), pad=9, shift=1)
    big = [torch.full((6, cols + 3), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    y, s, rstd = ra.rms_norm(x, None, residual=r, stats=True, out=big[0][:, 2:2 + cols], sum_out=big[1][:, 1:1 + cols])
    assert torch.equal(s, _sum(x, r))
    (want, _), (ey, _) = L.rms_forward(s, None, 1e-6)
    assert_within(y, want, rounded(dtype, want, ey), "y")
    assert (big[0][:, :2] == 7).all() and (big[0][:, 2 + cols:] == 7).all() and (big[1][:, :1] == 7).all() and (big[1][:, 1 + cols:] == 7).all()
    _check_fp8(*ra.rms_norm_fp8(x, group=128), x, None, 1e-6, 128, "fp8")
    grads = ra.rms_norm_backward(x, s, rstd, dsum=r)
    want, bound = L.rms_backward(x, s, rstd, None, r)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight")):
        assert_within(a, c, e, what)
    # each gradient alone is the same gradient
    assert torch.equal(ra.rms_norm_backward(x, s, rstd, dsum=r, dweight=False)[0], grads[0])
    assert torch.equal(ra.rms_norm_backward(x, s, rstd, dsum=r, dx=False)[1], grads[1])


@pytest.mark.parametrize("cols", [5, 50, 700, 5000, 18000])
def test_rms_norm_in_place_and_special_rows(cols):
    g = _gen("rms special", cols)
    x, r = _rand(g, (6, cols), F32), _rand(g, (6, cols), F32)
    x[1], r[1] = 0.0, 0.0
    x[2, cols // 2] = NAN
    x[3, 0] = INF
    x[4] *= 1e-30
    r[4] *= 1e-30
    w = _rand(g, (cols,), F32)
    y, s, rstd = ra.rms_norm(x, w, residual=r, stats=True)
    assert (y[1] == 0).all() and y[2].isnan().all() and y[3, 0].isnan() and (y[3, 1:] == 0).all() and y[4:].isfinite().all()
    for y_at, s_at in (("x", "r"), ("r", "x"), ("x", None), (None, "r"), (None, "x")):
        t = {"x": x.clone(), "r": r.clone(), None: None}
        y2, s2 = ra.rms_norm(t["x"], w, residual=t["r"], out=t[y_at], sum_out=t[s_at])
        assert torch.equal(s2.view(torch.int32), s.view(torch.int32)) and torch.equal(y2.view(torch.int32), y.view(torch.int32)), (y_at, s_at)
    t = s.clone()
    assert ra.rms_norm(t, w, out=t).data_ptr() == t.data_ptr() and torch.equal(t.view(torch.int32), y.view(torch.int32))
    for group in (None, 128):
        q, scale = ra.rms_norm_fp8(s, w, group=group)
        q = q.float()
        assert (q[1] == 0).all() and (scale[1] == 2.0 ** -126).all()
        assert q[2].isnan().all() and scale[2].isnan().all() and scale[3, 0].isnan() and q[4:].isfinite().all()


def test_rms_norm_many_rows_dims_and_none():
    g = _gen("rms rows")
    x, w = _rand(g, (3, 1500, 96), BF16), _rand(g, (96,), BF16)
    y, rstd = ra.rms_norm(x, w, stats=True)
    assert y.shape == x.shape and rstd.shape == (3, 1500)
    (want, _), (ey, _) = L.rms_forward(x, w, 1e-6)
    assert_within(y, want, rounded(BF16, want, ey), "y")
    q, scale = ra.rms_norm_fp8(x, w, group=128)
    assert q.shape == x.shape and scale.shape == (3, 1500, 1)
    dy = _rand(g, x.shape, BF16)
    grads = ra.rms_norm_backward(dy, x, rstd, w)
    want, bound = L.rms_backward(dy, x, rstd, w, None)
    for a, c, e, what in zip(grads, want, bound, ("dx", "dweight")):
        assert_within(a, c, e, what)
    e = torch.empty(0, 96, dtype=BF16, device="cuda")
    y, s, rstd = ra.rms_norm(e, w, residual=e, stats=True)
    assert y.shape == s.shape == (0, 96) and rstd.shape == (0,)
    assert (ra.rms_norm_backward(e, e, rstd, w)[1] == 0).all()


def test_rms_gradients_against_differences():
    g = _gen("rms differences")
    x, w, dy, ds = _rand(g, (7, 300), F32), _rand(g, (300,), F32), _rand(g, (7, 300), F32), _rand(g, (7, 300), F32)
    rstd = ra.rms_norm(x, w, 1e-3, stats=True)[1]
    dx, dw = (t.double().cpu() for t in ra.rms_norm_backward(dy, x, rstd, w, dsum=ds))
    x, w, dy, ds = (t.double().cpu() for t in (x, w, dy, ds))
    value = lambda x, w: (x / (x.square().mean(-1, keepdim=True) + 1e-3).sqrt() * w * dy).sum() + (x * ds).sum()  # noqa: E731
    for got, at in ((dx, 0), (dw, 1)):
        step = torch.randn(got.shape, generator=g, dtype=torch.float64) * 1e-5
        slope = (value(x + step, w) - value(x - step, w) if at == 0 else value(x, w + step) - value(x, w - step)) / 2
        assert abs(slope - (got * step).sum()) <= 1e-5 * (got.abs() * step.abs()).sum(), at


# ------------------------------------------------------------------- dropout
DROP = [(1, 1), (3, 7), (1, 64), (17, 8), (5, 513), (33, 1001), (600, 40), (2, 4096), (3, 20000), (1, 70001)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", DROP)
def test_dropout(rows, cols, dtype):
    g = _gen("dropout", rows, cols, dtype)
    x, r = _rand(g, (rows, cols), dtype), _rand(g, (rows, cols), dtype)
    for p, seed, offset in ((0.1, 1, 0), (0.5, (1 << 64) - 1, (1 << 64) - 1), (0.25, 0x123456789ABCDEF0, 5 << 32)):
        keep = L.kept(rows, cols, p, seed, offset)
        for residual in (None, r):
            y = ra.dropout(x, p, seed, offset, residual=residual)
            want, bound = L.dropped(x, keep, p, residual)
            assert_within(y, want, bound, (p, seed))
            if residual is None:
                assert torch.equal((y != 0).cpu(), keep & (x != 0).cpu())
        assert torch.equal(ra.dropout_backward(x, p, seed, offset), ra.dropout(x, p, seed, offset))


def test_the_generator_is_the_published_one():
    """Known answers of Philox4x32-10 (the paper's test vectors): a counter and
    key of zeros, of ones, and of the digits of pi, here in the oracle; the GPU's
    masks equal the oracle's above."""
    for counter, key, want in (
            ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0], [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        assert L.philox(np.array(counter), key).tolist() == want


@pytest.mark.parametrize("dtype", TYPES)
def test_dropout_extremes_and_what_is_dropped(dtype):
    g = _gen("dropout extremes", dtype)
    x, r = _rand(g, (9, 301), dtype), _rand(g, (9, 301), dtype)
    assert torch.equal(ra.dropout(x, 0.0, 3), x) and torch.equal(ra.dropout(x, 2.0 ** -18, 3), x)
    assert (ra.dropout(x, 1.0, 3) == 0).all() and torch.equal(ra.dropout(x, 1.0, 3, residual=r), r)
    keep = L.kept(9, 301, 0.5, 3).cuda()
    for bad in (NAN, INF, -INF):      # nothing of a dropped value is left
        assert torch.equal(ra.dropout(torch.where(keep, x, torch.full_like(x, bad)), 0.5, 3, residual=r), ra.dropout(x, 0.5, 3, residual=r))


@pytest.mark.parametrize("dtype", TYPES)
def test_dropout_parts_of_an_array_have_its_mask(dtype):
    """What a rank that holds some rows, or some columns, computes; strided and
    in place as well."""
    g = _gen("dropout parts", dtype)
    x, r = _rand(g, (40, 333), dtype), _rand(g, (40, 333), dtype)
    whole = ra.dropout(x, 0.3, 11, 4, residual=r)
    for lo, hi in ((0, 13), (13, 14), (14, 40)):
        assert torch.equal(ra.dropout(x[lo:hi], 0.3, 11, 4, residual=r[lo:hi], first_row=lo), whole[lo:hi])
    for lo, hi in ((0, 8), (8, 160), (160, 333)):
        assert torch.equal(ra.dropout(x[:, lo:hi], 0.3, 11, 4, residual=r[:, lo:hi], first_col=lo), whole[:, lo:hi])
    assert torch.equal(ra.dropout(_inside(x), 0.3, 11, 4, residual=_inside(r, 9, 1)), whole)
    t = x.clone()
    assert ra.dropout(t, 0.3, 11, 4, residual=r, out=t).data_ptr() == t.data_ptr() and torch.equal(t, whole)
    t = r.clone()
    assert torch.equal(ra.dropout(x, 0.3, 11, 4, residual=t, out=t), whole)
    last = (1 << 32) - 40
    assert_within(ra.dropout(x, 0.3, 11, first_row=last), *L.dropped(x, L.kept(40, 333, 0.3, 11, 0, last), 0.3), "last rows")
    assert ra.dropout(x[:0], 0.3, 11).shape == (0, 333)


def test_dropout_offset_in_memory_and_captured():
    """A captured call reads its offset at every replay."""
    g = _gen("dropout capture")
    x = _rand(g, (64, 1000), BF16)
    offset = torch.zeros(1, dtype=torch.int64, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        ra.dropout(x, 0.4, 9, offset)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            y = ra.dropout(x, 0.4, 9, offset)
    for n in (0, 1, (5 << 32) + 7, 1):
        with torch.cuda.stream(st):
            offset.fill_(n)
            graph.replay()
            st.synchronize()
        assert torch.equal(y, ra.dropout(x, 0.4, 9, n)), n
    for bad in (offset.int(), offset.cpu(), torch.zeros(2, dtype=torch.int64, device="cuda")):
        with pytest.raises(ra.RingarError):
            ra.dropout(x, 0.4, 9, bad)


def test_dropout_share_that_is_kept():
    """2^24 numbers: the kept share is within 6 standard deviations of 1 - p, and
    so is every one of the eight places of a block."""
    x = torch.ones(1 << 11, 1 << 13, device="cuda")
    for p in (0.1, 0.5):
        keep = (ra.dropout(x, p, 77) != 0).double()
        q = 1 - L.threshold(p) / 65536
        for t in (keep, *(keep[:, i::8] for i in range(8))):
            assert abs(float(t.mean()) - q) <= 6 * (q * (1 - q) / t.numel()) ** 0.5


def test_more_than_2_31_values():
    n = (1 << 31) // 4096 + 3
    x = torch.ones(n, 4096, dtype=F16, device="cuda")
    y = ra.dropout(x, 0.5, 5)
    for lo in (0, n - 4):
        assert torch.equal(y[lo:lo + 4].cpu() != 0, L.kept(4, 4096, 0.5, 5, 0, lo))
    y, rstd = ra.rms_norm(x, stats=True, out=y)
    one = ra.rms_norm(x[:1])
    assert torch.equal(y[-1:], one) and torch.equal(y[n // 2:n // 2 + 1], one) and (rstd == rstd[0]).all()
    q, scale = ra.rms_norm_fp8(x, group=128)
    assert torch.equal(q[-1].view(torch.uint8), q[0].view(torch.uint8)) and (scale == scale[0]).all()
