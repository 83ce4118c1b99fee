"""Which sources make a committed memory-traffic record stale (CPU)."""
import os
import shutil

import bench


def test_a_traffic_record_goes_by_the_collectives_kernels(tmp_path, monkeypatch):
    csrc = os.path.join("ring_allreduce_reduce_amd", "csrc")
    shutil.copytree(os.path.join(bench.ROOT, csrc), tmp_path / csrc)
    before = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == before

    def append(name, text):
        with open(tmp_path / csrc / name, "a") as f:
            f.write(text)

    # another operator's kernels, a host file, a comment
    append("norm_kernels.hip", "\nint other;\n")
    append("gemm_tile.h", "\nint other;\n")
    append("new_operator.hip", "int other;\n")
    append("ringar.cpp", "\nint other;\n")
    append("ring_launch.hip", "\n// a comment\n")
    assert bench.kernel_source_hash() == before
    seen = {before}
    for name in ("ring_kernel_impl.h", "ring_launch.hip", "tree_f32.hip", "captured_i8.hip", "ring_geometry.h"):
        append(name, "\nint changed;\n")
        assert bench.kernel_source_hash() not in seen, name
        seen.add(bench.kernel_source_hash())
