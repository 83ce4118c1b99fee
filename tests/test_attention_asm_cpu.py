"""The attention kernels' loads into LDS keep the hardware's wait states
(compiled for gfx950 here, read as assembly): the compiler looks after neither
before asm."""
import os
import re

import pytest

from ring_allreduce_reduce_amd import _build
from test_block_asm_cpu import _listing, _loads_to_lds, _scalars


@pytest.mark.parametrize("unit", ["attn_fwd_bf16.hip", "attn_bwd_bf16.hip", "attn_fwd_f32.hip", "attn_bwd_f32.hip"])
def test_wait_states_before_loads_into_lds(unit, tmp_path):
    """A wait state after m0 is set, and no scalar that a load takes written by a
    vector instruction within five wait states."""
    lines = _listing(tmp_path, os.path.join(_build.CSRC, unit))
    loads = [i for i, line in enumerate(lines) if _loads_to_lds(line)]
    assert loads
    for at in loads:
        first, last = map(int, re.search(r"s\[(\d+):(\d+)\]", lines[at]).groups())
        taken = {"m0"} | {f"s{i}" for i in range(first, last + 1)}
        waited, i = 0, at - 1
        while i >= 0 and waited < 5:
            line = lines[i]
            written = _scalars(line.split(None, 1)[1].split(",")[0]) if " " in line or "\t" in line else set()
            if line.startswith("s_nop"):
                waited += int(line.split()[1], 0) + 1
            else:
                assert not (line.startswith("v_") and written & taken), (line, lines[at])
                assert not ("m0" in written and waited == 0), (line, lines[at])
                waited += 1
            i -= 1


@pytest.mark.parametrize("unit", ["attn_fwd_bf16.hip", "attn_bwd_bf16.hip"])
def test_the_kernels_keep_their_registers(unit, tmp_path):
    """No vector register spilled: a spill's access waits for the loads into LDS
    that are on their way."""
    lines = _listing(tmp_path, os.path.join(_build.CSRC, unit))
    assert not [line for line in lines if line.startswith("scratch_")]
