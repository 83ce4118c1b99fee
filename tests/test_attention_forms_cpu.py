"""The plan gives attention_forms' sizes to the kernels that they are named for
(CPU, over a stand-in for the HIP runtime): a change of the plan's constants
cannot leave a kernel without its numerical tests."""
import pytest

import host_runtime
from attention_forms import CASES, F16, F32, tile_keys
from test_layer_host_cpu import MAKE


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return host_runtime.build(tmp_path_factory.mktemp("fake"))


def test_the_sizes_reach_the_kernels_of_many_rows(fake):
    import textwrap
    cases = []
    for dtype, waves, parts, b, lq, n, h, kv, d in CASES:
        wide = dtype == F32
        columns = 64 if d <= 64 else 96 if wide and d <= 96 else 128
        kernel = f"Li{columns}ELi{tile_keys(dtype)}ELi{waves[0]}ELi{waves[1]}E"
        cases.append(((b, lq, n, h, kv, d), 4 if wide else 2 if dtype == F16 else 3, kernel, parts))
    host_runtime.run(fake, textwrap.dedent(MAKE) + textwrap.dedent(f"""
        for shape, dtype, kernel, parts in {cases!r}:
            for lengths in (False, True):
                got = [l[0] for l in run("ringar_cross_attention", attention(*shape, dtype=dtype, lengths=lengths)) if "clear" not in l[0]]
                assert "attn_forward" in got[0] and kernel in got[0], (shape, dtype, got)
                assert [("join" in name) for name in got[1:]] == [True] * parts, (shape, dtype, got)
    """))
    # every kernel of many rows is among them
    assert len({c[2] for c in cases if c[1] == 3}) == 4 and len({c[2] for c in cases if c[1] == 4}) == 4
