"""The products' loads into LDS tell the compiler which register they change
(compiled for gfx950 here, read as assembly)."""
import os
import re
import subprocess

import pytest

from ring_allreduce_reduce_amd import _build

SOURCE = r"""
#include "gemm_tile.h"
using namespace ringar;
// a load of the tile's between two of the compiler's own to one LDS address,
// which it holds in m0
extern "C" __global__ void probe(const void* p, float* out) {
  __shared__ __attribute__((aligned(1024))) char lds[2][1024];
  Operand<float, true, 8, 1> op;
  op.start(p, 0, 1024, 128);
  op.offsets(128, 0, threadIdx.x, [](int r) { return r * 128; });
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p, (RINGAR_LDS void*)lds[1], 4, 0, 0);
  op.next_step();
  op.load(0, lds[0], 0);
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p, (RINGAR_LDS void*)lds[1], 4, 256, 0);
  wait_loads<>();
  out[threadIdx.x] = *(float*)(lds[0] + threadIdx.x * 4) + *(float*)(lds[1] + threadIdx.x * 4);
}
"""


def _listing(tmp_path, src=None):
    out = tmp_path / "listing.s"
    if src is None:
        src = tmp_path / "probe.hip"
        src.write_text(SOURCE)
    cmd = [_build._hipcc(), *_build.HIPCC_FLAGS, "-I", _build.CSRC, "-I", os.path.join(_build.ROOT, "include"), "-x", "hip",
           "--cuda-device-only", "-S", str(src), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    # the instructions, without labels, directives and comments
    lines = [line.split(";")[0].strip() for line in out.read_text().splitlines() if line.startswith("\t")]
    return [line for line in lines if line and not line.startswith(".")]


def _sets_m0(line):
    return bool(re.match(r"\S+ m0,", line))


def _loads_to_lds(line):
    return bool(re.match(r"buffer_load_\S+ .*\blds\b|global_load_lds", line))


def test_m0_is_set_again_after_a_load_into_lds(tmp_path):
    kinds = ["set" if _sets_m0(line) else "load" for line in _listing(tmp_path) if _sets_m0(line) or _loads_to_lds(line)]
    assert kinds.count("load") == 3
    for i, k in enumerate(kinds):
        assert k == "set" or kinds[i - 1] == "set", kinds


def test_an_instruction_lies_between_m0_and_the_load_that_takes_it(tmp_path):
    """The hardware needs a wait state there, which the compiler adds before
    its own loads only."""
    lines = _listing(tmp_path)
    after = [lines[i + 1] for i, line in enumerate(lines) if _sets_m0(line)]
    assert after and not any(_loads_to_lds(line) for line in after), after


@pytest.mark.parametrize("unit", ["gemm_nt_f32.hip", "gemm_nn_bf16.hip", "gemm_tn_bf16.hip"])
def test_loads_into_lds_of_the_products(unit, tmp_path):
    """In the kernels as built: a wait state after m0, and no scalar that a
    load takes written by a vector instruction within five wait states (the
    compiler looks after neither before asm)."""
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


def _scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand.strip())
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    return {operand.strip()} if re.match(r"(s\d+|m0)$", operand.strip()) else set()
