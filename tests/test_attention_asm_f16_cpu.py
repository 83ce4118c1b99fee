"""The fp16 attention kernels, which differ from the other types' in how they hold
P and dS, keep the hardware's wait states and their registers too (compiled for
gfx950 here, read as assembly)."""
import pytest

from test_attention_asm_cpu import test_the_kernels_keep_their_registers as registers
from test_attention_asm_cpu import test_wait_states_before_loads_into_lds as wait_states


@pytest.mark.parametrize("unit", ["attn_fwd_f16.hip", "attn_bwd_f16.hip"])
def test_fp16(unit, tmp_path):
    wait_states(unit, tmp_path)
    registers(unit, tmp_path)
