"""Attention's plan goes by sizes and types: lengths, which only the GPU knows, do not
change it (CPU, over a stand-in for the HIP runtime)."""
import textwrap

import pytest

import host_runtime
from test_layer_host_cpu import MAKE


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return host_runtime.build(tmp_path_factory.mktemp("fake"))


def test_lengths_do_not_change_the_plan(fake):
    host_runtime.run(fake, textwrap.dedent(MAKE) + textwrap.dedent("""
        count = 0
        for dtype in (2, 3, 4):
            for shape in ((53, 1, 6402, 2, 1, 128), (26, 1, 3968, 2, 2, 128), (5, 1, 8014, 18, 9, 40), (10, 11, 3087, 16, 4, 64), (1, 2, 7936, 24, 6, 80),
                          (32, 1, 2048, 32, 8, 128), (3, 333, 1501, 20, 20, 64), (8, 1024, 2048, 16, 16, 128), (15, 1, 7095, 1, 1, 64)):
                for back in (False, True):
                    name = "ringar_cross_attention" + "_backward" * back
                    got = [run(name, attention(*shape, dtype=dtype, back=back, lengths=l)) for l in (False, True, False)]
                    assert got[1] == got[2], (shape, dtype, back)          # (the first allocates)
                    count += 1
        assert count == 54
    """))
