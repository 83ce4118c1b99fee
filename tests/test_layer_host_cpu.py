"""The host side of the root-mean-square norm, dropout and cross attention, over a
stand-in for the HIP runtime that records launches and allocations (CPU)."""
import pytest

import host_runtime

MAKE = """
    from test_layer_abi_cpu import A, att, att_back, drop, rms, rms_back, strides
    far = [(i + 1) << 46 for i in range(12)]
    def attention(b, lq, n, h, kv, d, dtype=3, back=False, lengths=True, **kw):
        qs, ks = strides(lq * h * d, h * d, d), strides(n * kv * d, kv * d, d)
        a = dict(dtype=dtype, batch=b, queries=lq, keys=n, heads=h, kv_heads=kv, head_dim=d, scale=0.1, q_strides=qs, k_strides=ks, v_strides=ks,
                 y_strides=qs, key_lengths=far[10] if lengths else None, lse=far[9])
        a.update(zip(("q", "k", "v", "y"), far))
        if back:
            a.update(zip(("dy", "dq", "dk", "dv"), far[4:8]), dy_strides=qs)
        return (att_back if back else att)(**{**a, **kw})
    def run(name, args, stream=0x1000):
        fake.fake_reset()
        code = on(name, args, stream)
        assert code == 0, (name, code, ra.ringar_last_error())
        return launches()
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return host_runtime.build(tmp_path_factory.mktemp("fake"))


def _run(fake, code):
    import textwrap
    host_runtime.run(fake, textwrap.dedent(MAKE) + textwrap.dedent(code))


def test_launches_and_workspaces(fake):
    """One launch where nothing is split, a second for the parts; the backward
    pass's statistics and parts in the stream's one workspace."""
    _run(fake, """
        got = run("ringar_cross_attention", attention(8, 1024, 2048, 16, 16, 128))
        assert len(got) == 1 and got[0][1][0] == 8 * 16 * 8 and fake.fake_mallocs() == 0
        got = run("ringar_cross_attention", attention(1, 1, 16384, 32, 8, 128))
        assert [("join" in l[0]) for l in got if "clear" not in l[0]] == [False, True] and fake.fake_mallocs() == 1
        got = run("ringar_cross_attention_backward", attention(8, 1024, 2048, 16, 16, 128, back=True))
        assert ["attn_dq" in l[0] for l in got if "clear" not in l[0]] == [True, False]
        got = run("ringar_cross_attention_backward", attention(8, 1024, 2048, 16, 16, 128, back=True, dq=None))
        assert "attn_delta" in got[0][0] and "attn_dkv" in got[1][0] and len(got) == 2 and fake.fake_mallocs() == 0
        got = run("ringar_cross_attention_backward", attention(1, 64, 2048, 2, 2, 64, back=True))
        assert sum("attn_join" in l[0] for l in got) >= 1
        assert len(run("ringar_rms_norm", rms())) == 1 and len(run("ringar_dropout", drop())) == 1
        assert len(run("ringar_rms_norm_backward", rms_back(rows=1000))) == 2 and len(run("ringar_rms_norm_backward", rms_back())) == 1
    """)


def test_capture_needs_a_call_of_the_same_shape_first(fake):
    _run(fake, """
        args = attention(1, 1, 16384, 32, 8, 128)
        fake.fake_capture(1)
        assert on("ringar_cross_attention", args, 0x2000) == ra.INVALID_USAGE and launches() == []
        assert on("ringar_cross_attention_backward", attention(2, 8, 64, 2, 2, 64, back=True), 0x2000) == ra.INVALID_USAGE
        assert on("ringar_cross_attention", attention(8, 1024, 2048, 16, 16, 128), 0x2000) == 0       # needs no workspace
        fake.fake_capture(0)
        run("ringar_cross_attention", args, 0x2000)
        fake.fake_capture(1)
        assert on("ringar_cross_attention", args, 0x2000) == 0
    """)


def test_an_error_of_a_launch_is_the_calls(fake):
    _run(fake, """
        calls = [("ringar_cross_attention", attention(1, 1, 16384, 32, 8, 128), b"attn_forward_join"), ("ringar_rms_norm", rms(), b"rms_forward"),
                 ("ringar_cross_attention_backward", attention(2, 8, 64, 2, 2, 64, back=True), b"attn_dkv"), ("ringar_dropout", drop(), b"dropout"),
                 ("ringar_rms_norm_backward", rms_back(rows=1000), b"col_sum")]
        for name, args, kernel in calls:
            fake.fake_fail(kernel)
            assert on(name, args, 0x1000) == ra.DEVICE and fake.hipGetLastError() == 0, name
            fake.fake_stale_error(2)
            assert on(name, args, 0x1000) == 0 and fake.hipGetLastError() == 2, name
    """)


def test_sizes_at_the_limits(fake):
    """Whatever the sizes: launches within the runtime's limits, or a refusal."""
    _run(fake, """
        big = (1 << 31) - 1025
        for kw in (dict(rows=big, cols=8), dict(rows=1, cols=big), dict(rows=1 << 20, cols=20000)):
            c = kw["cols"]
            for out in (0, 1, 2):
                run("ringar_rms_norm", rms(dtype=3, out=out, scale=far[6], x=far[0], residual=far[1], weight=far[2], sum=far[3], y=far[4], rstd=far[5],
                                           ldx=c, ldr=c, lds=c, ldy=c, **kw))
            if kw["rows"] * c < 1 << 34:
                run("ringar_rms_norm_backward", rms_back(dy=far[0], x=far[1], rstd=far[2], weight=far[3], dsum=far[4], dx=far[5], dweight=far[6],
                                                         lddy=c, ldx=c, ldds=c, lddx=c, **kw))
            run("ringar_dropout", drop(x=far[0], residual=far[1], y=far[2], more_offset=far[3], ldx=c, ldr=c, ldy=c, **kw))
        for shape in ((1, big, 4, 1, 1, 8), (1, 1, big, 1, 1, 8), (4096, 1, 64, 512, 512, 8), (1 << 20, 1, 4, 8, 8, 64), (1, 1 << 24, 64, 64, 1, 64)):
            run("ringar_cross_attention", attention(*shape))
        for shape in ((1 << 20, 1, 4, 64, 64, 64), (1 << 22, 300, 4, 8, 8, 64)):
            assert on("ringar_cross_attention", attention(*shape), 0x1000) == ra.INVALID_USAGE, shape
            assert on("ringar_cross_attention_backward", attention(*shape, back=True), 0x1000) == ra.INVALID_USAGE, shape
    """)
