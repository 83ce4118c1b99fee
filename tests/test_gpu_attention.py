"""Cross attention on the GPU against its plain fp64 form: types, head
layouts, lengths from one key to long ones, shared key heads, masks that leave
a row empty, what lies past a length, captured calls and gradients."""
import math
import zlib

import pytest
import torch

import layer_refs as L
import ring_allreduce_reduce_amd as ra
from block_refs import assert_within

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [F32, F16, BF16]
NAN, INF = float("nan"), float("inf")


def _gen(*key):
    print("case", *key, flush=True)
    g = torch.Generator()
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def _rand(g, shape, dtype, layout="rows", fill=None):
    """Random (batch, rows, heads, dim): rows first, heads first, or one of two in a wider array of `fill`."""
    b, n, h, d = shape
    if layout == "heads":
        return torch.randn(b, h, n, d, generator=g).to(dtype).cuda().transpose(1, 2)
    t = torch.randn(shape, generator=g).to(dtype).cuda()
    if layout == "rows":
        return t
    pad = 16 // t.element_size()
    wide = torch.full((b, n + 1, 2, h, d + pad), NAN if fill is None else fill, dtype=dtype, device="cuda")
    v = wide[:, :n, 1, :, pad:]
    v.copy_(t)
    return v


def _lengths(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def _check(g, dtype, b, lq, n, h, kv, d, layout="rows", lengths=None, scale=None):
    q = _rand(g, (b, lq, h, d), dtype, layout)
    k, v = _rand(g, (b, n, kv, d), dtype, layout), _rand(g, (b, n, kv, d), dtype, layout)
    y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, scale=scale, stats=True)
    assert y.shape == q.shape and lse.shape == (b, h, lq) and lse.dtype == F32
    want, bound = L.attention(q, k, v, lengths, scale)
    assert_within(y, want[0], bound[0], "y")
    got = lse.double().cpu()
    empty = torch.isinf(want[1])
    assert torch.equal(got[empty], want[1][empty])
    assert ((got - want[1])[~empty].abs() <= bound[1][~empty]).all(), "lse"
    assert torch.equal(ra.cross_attention(q, k, v, key_lengths=lengths, scale=scale), y)
    dy = _rand(g, (b, lq, h, d), dtype, layout)
    grads = ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths, scale=scale)
    want, bound = L.attention_backward(dy, q, k, v, y, lse, lengths, scale)
    for a, c, e, what in zip(grads, want, bound, ("dq", "dk", "dv")):
        assert a.is_contiguous() and a.dtype == dtype
        assert_within(a, c, e, what)
    return q, k, v, y, lse, dy, grads


# batch, queries, keys, heads, key heads, head_dim
SIZES = [(1, 1, 1, 1, 1, 8), (1, 1, 5, 2, 2, 64), (2, 1, 31, 4, 1, 128), (1, 3, 32, 2, 2, 64), (1, 33, 33, 1, 1, 64), (2, 7, 64, 6, 2, 80),
         (1, 129, 65, 2, 1, 128), (1, 128, 100, 1, 1, 40), (3, 50, 257, 4, 2, 64), (1, 16, 700, 2, 1, 128), (2, 1, 2000, 8, 2, 64),
         (1, 200, 300, 7, 1, 72), (1, 31, 1023, 2, 2, 120), (1, 300, 1, 2, 2, 64), (2, 1, 513, 33, 1, 64), (1, 65, 129, 3, 3, 96)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,lq,n,h,kv,d", SIZES)
def test_sizes(b, lq, n, h, kv, d, dtype):
    _check(_gen("size", b, lq, n, h, kv, d, dtype), dtype, b, lq, n, h, kv, d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["heads", "inside"])
@pytest.mark.parametrize("b,lq,n,h,kv,d", [(2, 1, 300, 4, 2, 64), (3, 40, 140, 4, 2, 128), (2, 150, 70, 3, 3, 24)])
def test_layouts_and_lengths(b, lq, n, h, kv, d, layout, dtype):
    g = _gen("layout", b, lq, n, layout, dtype)
    _check(g, dtype, b, lq, n, h, kv, d, layout, _lengths(*[(n * (2 * i + 1)) // (2 * b) for i in range(b)]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq", [1, 40, 200])
def test_empty_sequences_and_lengths_out_of_range(lq, dtype):
    g = _gen("empty", lq, dtype)
    lengths = _lengths(0, 1, -5, 65, 1 << 30, 32)
    q, k, v, y, lse, dy, grads = _check(g, dtype, 6, lq, 96, 4, 2, 64, lengths=lengths.clamp(0, 96))
    y2, lse2 = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
    assert torch.equal(y2, y) and torch.equal(lse2, lse)
    assert (y[0] == 0).all() and (y[2] == 0).all() and (lse[0] == -INF).all()
    assert all((t[0] == 0).all() for t in grads)
    assert (grads[1][1, 1:] == 0).all() and (grads[2][3, 65:] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq", [1, 70])
def test_what_lies_past_a_length_does_not_matter(lq, dtype):
    """NaN, infinities and the type's limits there."""
    g = _gen("past", lq, dtype)
    lengths = _lengths(70, 1, 64)
    q, k, v = _rand(g, (3, lq, 4, 64), dtype), _rand(g, (3, 200, 2, 64), dtype), _rand(g, (3, 200, 2, 64), dtype)
    dy = _rand(g, (3, lq, 4, 64), dtype)
    y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
    grads = ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths)
    for bad in (NAN, INF, -INF, torch.finfo(dtype).min, torch.finfo(dtype).max):
        k2, v2 = k.clone(), v.clone()
        for i, n in enumerate(lengths.tolist()):
            k2[i, n:] = bad
            v2[i, n:] = bad
        y2, lse2 = ra.cross_attention(q, k2, v2, key_lengths=lengths, stats=True)
        assert torch.equal(y, y2) and torch.equal(lse, lse2), bad
        for a, b in zip(grads, ra.cross_attention_backward(dy, q, k2, v2, y, lse, key_lengths=lengths)):
            assert torch.equal(a, b), bad


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_and_infinity_stay_in_their_rows(dtype):
    g = _gen("nan", dtype)
    for lq in (1, 100):
        q, k, v = _rand(g, (2, lq, 3, 64), dtype), _rand(g, (2, 90, 3, 64), dtype), _rand(g, (2, 90, 3, 64), dtype)
        want = ra.cross_attention(q, k, v)
        q[0, 0, 1, 5] = NAN
        v[1, 40, 2, 7] = INF
        got = ra.cross_attention(q, k, v)
        assert got[0, 0, 1].isnan().all()
        assert (got[1, :, 2, 7] == INF).all()
        same = torch.ones_like(got, dtype=torch.bool)
        same[0, 0, 1] = False
        same[1, :, 2, 7] = False
        assert torch.equal(got[same], want[same])


@pytest.mark.parametrize("dtype", TYPES)
def test_scores_far_apart_and_far_from_zero(dtype):
    """Rising scores move the running maximum at every tile; scores of some
    hundreds, of either sign, stay finite and exact."""
    g = _gen("far", dtype)
    b, lq, n, h, d = 1, 40, 400, 1, 64
    q, k, v = (torch.zeros(b, r, h, d) for r in (lq, n, n))
    v = torch.randn(v.shape, generator=g)
    q[..., 0] = torch.linspace(-2, 2, lq)[None, :, None]
    k[..., 0] = torch.linspace(-300, 300, n)[None, :, None]
    q, k, v = (t.to(dtype).cuda() for t in (q, k, v))
    for scale in (0.01, 0.125, 1.0):
        y, lse = ra.cross_attention(q, k, v, scale=scale, stats=True)
        want, bound = L.attention(q, k, v, None, scale)
        assert_within(y, want[0], bound[0], "y")
        assert ((lse.double().cpu() - want[1]).abs() <= bound[1]).all()
        dy = _rand(g, (b, lq, h, d), dtype)
        grads = ra.cross_attention_backward(dy, q, k, v, y, lse, scale=scale)
        want, bound = L.attention_backward(dy, q, k, v, y, lse, None, scale)
        for a, c, e, what in zip(grads, want, bound, ("dq", "dk", "dv")):
            assert_within(a, c, e, what)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lq", [1, 150])
def test_scores_of_minus_infinity_before_very_low_ones(lq, dtype):
    """The first tiles have no finite score, the later ones scores near -1000:
    the row is that of the later ones alone."""
    g = _gen("infinite", lq, dtype)
    q, k, v = _rand(g, (1, lq, 1, 64), dtype), _rand(g, (1, 400, 1, 64), dtype), _rand(g, (1, 400, 1, 64), dtype)
    q[..., 0] = 100.0
    k[..., 0] = -80.0
    q[..., 1] = 2.0 ** 70
    k[..., 1] = 0.0
    k[:, :192, :, 1] = -2.0 ** 70
    y, lse = ra.cross_attention(q, k, v, stats=True)
    k = k[:, 192:].contiguous()
    q[..., 1] = 0.0
    want, bound = L.attention(q, k, v[:, 192:], None, None)
    assert_within(y, want[0], bound[0], "y")
    assert ((lse.double().cpu() - want[1]).abs() <= bound[1]).all() and (lse < -900).all()


def test_row_strides_up_to_the_largest():
    """128 rows of keys 2^24 - 16 bytes apart, and more than that refused."""
    g = _gen("pitch")
    for d in (64, 128):
        pitch = (1 << 23) - 8
        big = torch.zeros(130 * pitch + 4096, dtype=BF16, device="cuda")
        k, v = (big.as_strided((1, 130, 1, d), (0, pitch, 0, 1), at) for at in (0, 256))
        k.copy_(_rand(g, k.shape, BF16))
        v.copy_(_rand(g, v.shape, BF16))
        q, dy = _rand(g, (1, 33, 1, d), BF16), _rand(g, (1, 33, 1, d), BF16)
        y, lse = ra.cross_attention(q, k, v, stats=True)
        assert torch.equal(y, ra.cross_attention(q, k.contiguous(), v.contiguous()))
        for a, b in zip(ra.cross_attention_backward(dy, q, k, v, y, lse), ra.cross_attention_backward(dy, q, k.contiguous(), v.contiguous(), y, lse)):
            assert torch.equal(a, b)
        with pytest.raises(ra.RingarError):
            ra.cross_attention(q, big.as_strided((1, 100, 1, d), (0, 1 << 23, 0, 1)), v[:, :100])


def test_long_inputs_and_few_sequences():
    """Keys split over blocks, forward and backward."""
    for dtype, n in ((BF16, 20011), (F32, 9001)):
        g = _gen("long", dtype, n)
        _check(g, dtype, 1, 1, n, 8, 2, 128, lengths=_lengths(n - 3))
        _check(g, dtype, 2, 5, n // 8, 2, 1, 64, lengths=_lengths(n // 8, 77))


def test_keys_repeated_by_a_stride_of_zero():
    g = _gen("stride 0")
    q = _rand(g, (3, 20, 4, 64), BF16)
    k, v = _rand(g, (1, 50, 1, 64), BF16).expand(3, -1, 2, -1), _rand(g, (1, 1, 2, 64), BF16).expand(3, 50, -1, -1)
    y, lse = ra.cross_attention(q, k, v, stats=True)
    assert torch.equal(y, ra.cross_attention(q, k.contiguous(), v.contiguous()))
    dy = _rand(g, (1, 20, 1, 64), BF16).expand(3, -1, 4, -1)
    got = ra.cross_attention_backward(dy, q, k, v, y, lse)
    for a, b in zip(got, ra.cross_attention_backward(dy.contiguous(), q, k.contiguous(), v.contiguous(), y, lse)):
        assert torch.equal(a, b)


def test_out_flags_and_sizes_of_zero():
    g = _gen("flags")
    q, k, v = _rand(g, (2, 30, 4, 64), F16), _rand(g, (2, 60, 2, 64), F16), _rand(g, (2, 60, 2, 64), F16)
    y, lse = ra.cross_attention(q, k, v, stats=True)
    big = torch.full((2, 31, 4, 80), 7.0, dtype=F16, device="cuda")
    out = big[:, :30, :, 8:72]
    assert ra.cross_attention(q, k, v, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out, y) and (big[..., :8] == 7).all() and (big[..., 72:] == 7).all() and (big[:, 30] == 7).all()
    dy = _rand(g, q.shape, F16)
    grads = ra.cross_attention_backward(dy, q, k, v, y, lse)
    for i, name in enumerate(("dq", "dk", "dv")):
        flags = {n: n == name for n in ("dq", "dk", "dv")}
        alone = ra.cross_attention_backward(dy, q, k, v, y, lse, **flags)
        assert [t is None for t in alone] == [n != name for n in ("dq", "dk", "dv")]
        assert torch.equal(alone[i], grads[i])
    e = lambda *s: torch.empty(s, dtype=F16, device="cuda")  # noqa: E731
    y, lse = ra.cross_attention(q, k[:, :0], v[:, :0], stats=True)
    assert (y == 0).all() and (lse == -INF).all()
    dq, dk, dv = ra.cross_attention_backward(dy, q, k[:, :0], v[:, :0], y, lse)
    assert (dq == 0).all() and dk.shape == dv.shape == (2, 0, 2, 64)
    dq, dk, dv = ra.cross_attention_backward(e(2, 0, 4, 64), e(2, 0, 4, 64), k, v, e(2, 0, 4, 64), torch.empty(2, 4, 0, device="cuda"))
    assert (dk == 0).all() and (dv == 0).all() and dq.shape == (2, 0, 4, 64)
    assert ra.cross_attention(e(0, 3, 4, 64), e(0, 5, 2, 64), e(0, 5, 2, 64)).shape == (0, 3, 4, 64)


def test_refusals_on_tensors():
    g = _gen("refusals")
    q, k, v = _rand(g, (2, 3, 4, 64), BF16), _rand(g, (2, 9, 2, 64), BF16), _rand(g, (2, 9, 2, 64), BF16)
    lengths = _lengths(1, 2)
    wide = _rand(g, (2, 9, 2, 72), BF16)
    for call in (lambda: ra.cross_attention(q, k, v[:, :5]), lambda: ra.cross_attention(q, k[:1], v[:1]), lambda: ra.cross_attention(q[0], k, v),
                 lambda: ra.cross_attention(q, k.half(), v), lambda: ra.cross_attention(q, k, v.cpu()), lambda: ra.cross_attention(q[:, :, :3], k, v),
                 lambda: ra.cross_attention(q, k, v, key_lengths=lengths.long()), lambda: ra.cross_attention(q, k, v, key_lengths=lengths[:1]),
                 lambda: ra.cross_attention(q, k, v, key_lengths=lengths.cpu()), lambda: ra.cross_attention(q, k, v, out=q),
                 lambda: ra.cross_attention(q, k, v, scale=0), lambda: ra.cross_attention(q, wide[..., 1:65], v),
                 lambda: ra.cross_attention(q.transpose(1, 3), k, v), lambda: ra.cross_attention(q, k, v, out=torch.empty_like(q)[:, :2]),
                 lambda: ra.cross_attention_backward(q, q, k, v, q, torch.zeros(2, 4, 4, device="cuda"))):
        with pytest.raises(ra.RingarError):
            call()


def test_gradients_against_differences():
    """Central differences of the fp64 form at the kernel's operands: sum(dy y)
    changes by the gradients along random directions."""
    g = _gen("differences")
    q, k, v = _rand(g, (2, 20, 4, 32), F32), _rand(g, (2, 50, 2, 32), F32), _rand(g, (2, 50, 2, 32), F32)
    lengths = _lengths(50, 21)
    y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
    dy = _rand(g, q.shape, F32)
    grads = [t.double().cpu() for t in ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths)]
    base = [t.double().cpu() for t in (q, k, v)]

    def value(tensors):
        a, b, c = tensors
        s = L._heads(a, 4) @ L._heads(b, 4).transpose(2, 3) / math.sqrt(32)
        s = s.masked_fill((torch.arange(50)[None, :] >= lengths.cpu()[:, None])[:, None, None, :], -INF)
        out = (torch.softmax(s, -1) @ L._heads(c, 4)).transpose(1, 2)
        return (out * dy.double().cpu()).sum()

    for i in range(3):
        step = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        plus, minus = ([t + (e * h * step if j == i else 0) for j, t in enumerate(base)] for e in (1, -1))
        slope = (value(plus) - value(minus)) / (2 * h)
        along = (grads[i] * step).sum()
        # differences: h^2 times third derivatives (below 1e-6 here); gradients: fp32 sums of 50 terms
        assert abs(slope - along) <= 1e-5 * (grads[i].abs() * step.abs()).sum(), i


def test_captured_and_replayed():
    """A graph of forward and backward, replayed on new inputs between eager
    calls of its stream."""
    g = _gen("capture")
    st = torch.cuda.Stream()
    q, k, v = _rand(g, (2, 5, 4, 64), BF16), _rand(g, (2, 900, 2, 64), BF16), _rand(g, (2, 900, 2, 64), BF16)
    dy, lengths = _rand(g, q.shape, BF16), _lengths(900, 300)
    torch.cuda.synchronize()

    def both():
        y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
        return [y, lse, *ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths)]

    with torch.cuda.stream(st):
        both()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            outs = both()
    for i in range(3):
        with torch.cuda.stream(st):
            q.copy_(_rand(g, q.shape, BF16))
            lengths.copy_(_lengths(900 - 100 * i, 7 * i))
            want = [t.clone() for t in both()]
            graph.replay()
            st.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b), i


def test_another_stream():
    g = _gen("stream")
    st = torch.cuda.Stream()
    q, k, v = _rand(g, (2, 5, 4, 64), F16), _rand(g, (2, 900, 2, 64), F16), _rand(g, (2, 900, 2, 64), F16)
    want, lse = ra.cross_attention(q, k, v, stats=True)
    grads = ra.cross_attention_backward(want, q, k, v, want, lse)
    torch.cuda.synchronize()
    y, l2 = ra.cross_attention(q, k, v, stats=True, stream=st)
    again = ra.cross_attention_backward(y, q, k, v, y, l2, stream=st)
    st.synchronize()
    assert torch.equal(y, want) and torch.equal(l2, lse)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))


def test_strides_beyond_31_bits():
    """Sequences more than 2^31 values apart."""
    g = _gen("far apart")
    big = torch.empty((1 << 31) + (1 << 20), dtype=BF16, device="cuda")
    far = lambda at, n, h: big.as_strided((2, n, h, 64), ((1 << 31) + 4096, h * 64, 64, 1), at)  # noqa: E731
    q, k, v, y = far(0, 9, 4), far(1 << 14, 40, 2), far(1 << 15, 40, 2), far(1 << 16, 9, 4)
    for t in (q, k, v):
        t.copy_(_rand(g, t.shape, BF16))
    want = ra.cross_attention(q.contiguous(), k.contiguous(), v.contiguous())
    lse = ra.cross_attention(q, k, v, stats=True)[1]
    with pytest.raises(ra.RingarError):      # its span holds the others
        ra.cross_attention(q, k, v, out=y)
    assert torch.equal(ra.cross_attention(q, k, v), want)
    got = ra.cross_attention_backward(q, q, k, v, want, lse)
    for a, b in zip(got, ra.cross_attention_backward(q.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), want, lse)):
        assert torch.equal(a, b)
