"""Attention's kernels of many rows (attention_forms: which sizes reach them)
against the plain fp64 form: tiles shared by waves, groups of waves with unlike
numbers of tiles, partial last tiles, scores that rise past what a tile taken
without a look for its maximum may hold, and what must not be looked at.

The key heads do not touch each other: the fp64 form is that of the first and the
last key head and the query heads that share them."""
import zlib

import pytest
import torch

import layer_refs as L
import ring_allreduce_reduce_amd as ra
from attention_forms import BF16, CASES, F32, lengths_of, tile_keys
from block_refs import assert_within

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
each_case = pytest.mark.parametrize("dtype,waves,parts,b,lq,n,h,kv,d", CASES)


def _gen(*key):
    print("case", *key, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def _rand(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def _operands(g, dtype, b, lq, n, h, kv, d):
    return _rand(g, (b, lq, h, d), dtype), _rand(g, (b, n, kv, d), dtype), _rand(g, (b, n, kv, d), dtype)


def _lengths(dtype, n):
    return torch.tensor(lengths_of(dtype, n), dtype=torch.int32, device="cuda")


def _ends(t, heads):
    """The heads of the first and the last key head, of `heads` key heads."""
    each = t.shape[2] // heads
    return torch.cat((t[:, :, :each], t[:, :, -each:]), 2)


def _check_forward(q, k, v, y, lse, lengths, scale=None):
    kv = k.shape[2]
    want, bound = L.attention(*(_ends(t, kv) for t in (q, k, v)), lengths, scale)
    assert_within(_ends(y, kv), want[0], bound[0], "y")
    got = _ends(lse.transpose(1, 2), kv).transpose(1, 2).double().cpu()
    empty = torch.isinf(want[1])
    assert torch.equal(got[empty], want[1][empty])
    assert ((got - want[1])[~empty].abs() <= bound[1][~empty]).all(), "lse"


@each_case
def test_unlike_lengths(dtype, waves, parts, b, lq, n, h, kv, d):
    """Forward and backward; an empty sequence, one key, whole and partial tiles, groups without a tile of their own."""
    g = _gen("lengths", dtype, waves, parts, n, d)
    q, k, v = _operands(g, dtype, b, lq, n, h, kv, d)
    lengths = _lengths(dtype, n)
    y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
    _check_forward(q, k, v, y, lse, lengths)
    assert torch.equal(ra.cross_attention(q, k, v, key_lengths=lengths), y)
    dy = _rand(g, q.shape, dtype)
    grads = ra.cross_attention_backward(dy, q, k, v, y, lse, key_lengths=lengths)
    want, bound = L.attention_backward(*(_ends(t, kv) for t in (dy, q, k, v, y)), _ends(lse.transpose(1, 2), kv).transpose(1, 2), lengths)
    for a, c, e, what in zip(grads, want, bound, ("dq", "dk", "dv")):
        assert_within(_ends(a, kv), c, e, what)


@each_case
def test_all_keys_and_another_layout(dtype, waves, parts, b, lq, n, h, kv, d):
    g = _gen("all", dtype, waves, parts, n, d)
    q, k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in _operands(g, dtype, b, lq, n, h, kv, d))
    y, lse = ra.cross_attention(q, k, v, stats=True)
    _check_forward(q, k, v, y, lse, None)
    assert torch.equal(ra.cross_attention(q.contiguous(), k.contiguous(), v.contiguous()), y)


@each_case
def test_what_lies_past_a_length(dtype, waves, parts, b, lq, n, h, kv, d):
    g = _gen("past", dtype, waves, parts, n, d)
    q, k, v = _operands(g, dtype, b, lq, n, h, kv, d)
    lengths = _lengths(dtype, n)
    y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, stats=True)
    past = (torch.arange(n, device="cuda")[None] >= lengths[:, None])[:, :, None, None]
    for bad in (NAN, INF, torch.finfo(dtype).min):
        y2, lse2 = ra.cross_attention(q, k.masked_fill(past, bad), v.masked_fill(past, bad), key_lengths=lengths, stats=True)
        assert torch.equal(y, y2) and torch.equal(lse, lse2), bad


@each_case
def test_scores_that_rise_and_fall(dtype, waves, parts, b, lq, n, h, kv, d):
    """Scores along a slope (of either sign by the row) raise the running maximum
    at every tile or at none, single keys far above the others in a middle tile
    and in the last one, a score of minus infinity's size never."""
    g = _gen("rise", dtype, waves, parts, n, d)
    q, k, v = _operands(g, dtype, b, lq, n, h, kv, d)
    q *= 0.25
    q[..., 0] = torch.linspace(-2, 2, lq, device="cuda")[None, :, None]
    k[..., 0] = torch.linspace(-300, 300, n, device="cuda")[None, :, None]
    q[..., 1] = 1.0
    k[..., 1] = 0.0
    k[:, n // 2, :, 1] = 200.0
    k[:, n - 2, ::2, 1] = 400.0
    lengths = _lengths(dtype, n)
    for scale in (0.01, 0.125, 1.0):
        y, lse = ra.cross_attention(q, k, v, key_lengths=lengths, scale=scale, stats=True)
        _check_forward(q, k, v, y, lse, lengths, scale)


@each_case
def test_nan_stays_in_its_rows(dtype, waves, parts, b, lq, n, h, kv, d):
    g = _gen("nan", dtype, waves, parts, n, d)
    q, k, v = _operands(g, dtype, b, lq, n, h, kv, d)
    want = ra.cross_attention(q, k, v)
    q[0, lq - 1, h - 1, 5] = NAN
    v[1, n - 1, 0, 7] = INF
    got = ra.cross_attention(q, k, v)
    rows = torch.zeros_like(got, dtype=torch.bool)
    rows[0, lq - 1, h - 1] = True
    assert got[rows].isnan().all()
    high = torch.zeros_like(rows)
    high[1, :, :h // kv, 7] = True
    assert (got[high] == INF).all()
    assert torch.equal(got[~(rows | high)], want[~(rows | high)])


@pytest.mark.parametrize("dtype,waves,parts,b,lq,n,h,kv,d", [c for c in CASES if c[0] in (BF16, F32)])
def test_minus_infinity_before_very_low_scores(dtype, waves, parts, b, lq, n, h, kv, d):
    """The first tiles of every group of waves have no finite score, the later ones scores near -1000."""
    g = _gen("infinite", dtype, waves, parts, n, d)
    q, k, v = _operands(g, dtype, b, lq, n, h, kv, d)
    first = 2 * tile_keys(dtype)
    q[..., 0] = 100.0
    k[..., 0] = -10.0 * d ** 0.5
    q[..., 1] = 2.0 ** 70
    k[..., 1] = 0.0
    k[:, :first, :, 1] = -2.0 ** 70
    y, lse = ra.cross_attention(q, k, v, stats=True)
    q[..., 1] = 0.0
    _check_forward(q, k[:, first:], v[:, first:], y, lse, None)
    assert (lse < -900).all()
