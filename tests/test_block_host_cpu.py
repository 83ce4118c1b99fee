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
        fake.fake_fail(b"fill_u64")
        assert on("ringar_linear", args, 0x1000) == ra.DEVICE
        assert launches() == []
        fake.fake_stale_error(0)
        assert on("ringar_linear", args, 0x1000) == 0
        names = [l[0] for l in launches()]
        assert len(names) == 2 and "fill_u64" in names[0] and "gemm_rows" in names[1], names
        assert fake.fake_mallocs() == 2 and fake.fake_frees() == 1
    """)
