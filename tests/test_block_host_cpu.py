"""The host side of the block operators, over a stand-in for the HIP runtime
that records launches and allocations (CPU)."""
import pytest

import host_runtime


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return host_runtime.build(tmp_path_factory.mktemp("fake"))


def test_per_thread_streams_do_not_share_a_workspace(fake):
    """hipStreamPerThread (handle 2) names another stream in every host
    thread; the backward pass of a few rows with long columns needs a
    workspace."""
    host_runtime.run(fake, """
        import threading
        args = lambda: lin_back(rows=4, in_features=64, out_features=4096, lddy=4096, ldp=4096)
        def two_calls():
            codes.append((on("ringar_linear_backward", args(), 2), on("ringar_linear_backward", args(), 2)))
        codes = []
        B._fn("ringar_linear_backward")
        for n in (1, 2, 3):
            t = threading.Thread(target=two_calls)
            t.start()
            t.join()
            assert fake.fake_mallocs() == n, (n, fake.fake_mallocs())
        assert codes == [(0, 0)] * 3, codes
        # an ordinary stream is one for all threads
        fake.fake_reset()
        for _ in range(2):
            t = threading.Thread(target=lambda: codes.append(on("ringar_linear_backward", args(), 0x1000)))
            t.start()
            t.join()
        assert fake.fake_mallocs() == 1 and codes[3:] == [0, 0]
        assert ra.ringar_release() in (None, 0)
        assert fake.fake_frees() == 4
    """)


def test_a_workspace_whose_counters_were_not_cleared_is_not_used(fake):
    """The clearing launch fails once: the call is refused, and the next one
    allocates and clears again."""
    host_runtime.run(fake, """
        args = lin(rows=4, in_features=8192, out_features=64, ldx=8192, ldw=8192, ldy=64)
        fake.fake_fail(b"clear_words")
        assert on("ringar_linear", args, 0x1000) == ra.DEVICE
        assert launches() == []
        fake.fake_stale_error(0)
        assert on("ringar_linear", args, 0x1000) == 0
        names = [l[0] for l in launches()]
        assert len(names) == 2 and "clear_words" in names[0] and "gemm_rows" in names[1], names
        assert fake.fake_mallocs() == 2 and fake.fake_frees() == 1
    """)


def test_an_error_of_somebody_elses_call_is_not_the_operators(fake):
    """An error that another runtime call has left on the thread: every
    operator still runs, first use of the workspace included, and leaves it
    for whoever asks."""
    host_runtime.run(fake, """
        many = dict(rows=300, in_features=256, out_features=512)
        for name, args in (("ringar_layer_norm", norm()), ("ringar_layer_norm_backward", norm_back(rows=400)), ("ringar_linear", lin()),
                           ("ringar_gated_ffn", lin()), ("ringar_linear", lin(**many, ldx=256, ldw=256, ldy=512, ldp=512)),
                           ("ringar_linear_backward", lin_back()), ("ringar_gated_ffn_backward", lin_back(ldp=64)),
                           ("ringar_linear_backward", lin_back(**many, ldx=256, ldw=256, lddx=256, lddw=256, lddy=512, ldp=512))):
            fake.fake_stale_error(2)
            assert on(name, args, 0x1000) == 0, (name, ra.ringar_last_error())
            assert fake.hipGetLastError() == 2, name
    """)


def test_a_failed_call_leaves_no_error_behind(fake):
    host_runtime.run(fake, """
        fake.fake_fail(b"norm_forward")
        assert on("ringar_layer_norm", norm(), 0) == ra.DEVICE and fake.hipGetLastError() == 0
        assert on("ringar_layer_norm", norm(), 0) == 0
        # a workspace beyond the memory
        far = lin_back(rows=1 << 20, out_features=1 << 18, in_features=1 << 12, ldx=1 << 12, ldw=1 << 12, lddx=1 << 12, lddw=1 << 12,
                       lddy=1 << 18, ldp=1 << 18, **{k: (i + 1) << 46 for i, k in enumerate(("dy", "pre", "x", "weight", "dx", "dweight", "dbias"))})
        assert on("ringar_linear_backward", far, 0) == ra.DEVICE and fake.hipGetLastError() == 0
    """)


def test_launches_of_the_largest_sizes(fake):
    """A launch takes fewer than 2^32 threads along a dimension: sizes whose
    blocks exceed that run in several launches, or in blocks that loop."""
    host_runtime.run(fake, """
        far = {k: (i + 1) << 46 for i, k in enumerate(("x", "weight", "y", "dy", "pre", "dx", "dweight", "dbias", "mean", "rstd", "bias"))}

        def product(name, rows, k, n, wide=None, **kw):
            wide = wide or n
            a = dict(rows=rows, in_features=k, out_features=n, ldx=k, ldw=k, **kw)
            back = name.endswith("backward")
            keys = ("x", "weight", "dy", "pre", "dx", "dweight", "dbias") if back else ("x", "weight", "y", "pre", "bias")
            a.update({key: far[key] for key in keys if key not in kw})
            a.update(dict(lddx=k, lddw=k, lddy=n, ldp=wide) if back else dict(ldy=n, ldp=wide))
            return (lin_back if back else lin)(**a)

        def blocks_of(name, args, kernel):
            fake.fake_reset()
            code = on(name, args, 0x1000)
            assert code == 0, (name, ra.ringar_last_error())
            found = [l for l in launches() if kernel in l[0]]
            assert found, (name, kernel, launches())
            return sum(l[1][0] * l[1][1] for l in found)

        big = 1 << 27
        # a few rows, 16 (gated: 8) columns a block
        assert blocks_of("ringar_linear", product("linear", 1, 8, big + 20, dtype=4), "gemm_rows") == big // 16 + 2
        assert blocks_of("ringar_gated_ffn", product("gated", 2, 8, big // 2 + 20, big + 40, dtype=4), "gemm_rows") == big // 16 + 3
        # tiles of 64 x 64
        for k in (8, 7):
            got = blocks_of("ringar_linear", product("linear", 1 << 30, k, 8), "gemm_tile")
            assert got == 1 << 24, got
        assert blocks_of("ringar_linear_backward", product("linear_backward", 1 << 30, 8, 8, act=0, dbias=None, dweight=None),
                         "gemm_") == 1 << 24
        blocks_of("ringar_linear_backward", product("linear_backward", 1 << 30, 8, 8, act=0), "gemm_")
        blocks_of("ringar_linear_backward", product("linear_backward", 20, 8, 1 << 29, act=4), "gemm_")
        # copies of odd rows
        blocks_of("ringar_linear", product("linear", 1 << 28, 129, 1001, pre=None), "gemm_tile")
        # parts of a few rows' dx
        blocks_of("ringar_linear_backward", product("linear_backward", 4, big, 520, act=4), "")
        blocks_of("ringar_linear_backward", product("linear_backward", 1, big, 520, act=4), "few_join")
        # rows beyond the registers, and their parameters' gradients
        rows, cols = 5000000, 16400
        norms = {k: far[k] for k in ("x", "weight", "bias", "mean", "rstd")}
        blocks_of("ringar_layer_norm", norm(rows=rows, cols=cols, ldx=cols, ldy=cols, y=far["y"], **norms), "norm_forward_long")
        del norms["bias"]
        for rows, cols in ((rows, cols), (3, 1 << 29)):
            blocks_of("ringar_layer_norm_backward", norm_back(rows=rows, cols=cols, ldx=cols, lddy=cols, lddx=cols, dy=far["dy"], dx=far["dx"],
                      dweight=far["dweight"], dbias=far["dbias"], **norms), "col_sum")
    """)


def test_which_products_of_few_rows_stream_the_weight(fake):
    """The rule's corners, as measured: 16-bit tiles take many weight rows
    with a short k or with more than 8 rows; fp32 streams all of them."""
    host_runtime.run(fake, """
        far = {k: (i + 1) << 46 for i, k in enumerate(("x", "weight", "y", "bias"))}
        def streams(dtype, rows, k, n, gated=False, pad=0):
            fake.fake_reset()
            args = lin(dtype=dtype, rows=rows, in_features=k, out_features=n, ldx=k + pad, ldw=k + pad, ldy=n, pre=None, **far)
            assert on("ringar_gated_ffn" if gated else "ringar_linear", args, 0x1000) == 0
            return any("gemm_rows" in l[0] for l in launches())
        for rows, k, n, pad, want in ((1, 4096, 4096, 0, 1), (16, 4096, 4096, 0, 1), (17, 4096, 4096, 0, 0), (16, 1024, 8192, 0, 1),
                                      (16, 2048, 12288, 0, 1), (4, 1024, 12288, 0, 0), (4, 1032, 16384, 0, 1), (8, 4096, 20480, 0, 1),
                                      (9, 4096, 20480, 0, 0), (4, 1023, 16384, 0, 1), (4, 1024, 16384, 1, 1), (1, 7, 4096, 0, 0)):
            assert streams(3, rows, k, n, pad=pad) == bool(want), (rows, k, n, pad)
            assert streams(2, rows, k, n // 2, True, pad) == bool(want), (rows, k, n, pad)
        for rows, k, n, want in ((16, 4096, 65536, 1), (16, 512, 65536, 1), (17, 512, 65536, 0), (9, 4095, 20480, 1), (1, 3, 64, 0), (1, 4, 64, 1)):
            assert streams(4, rows, k, n) == bool(want), (rows, k, n)
    """)
