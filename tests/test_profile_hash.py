"""CPU: a change of any source that the profiled kernels or their launches are built from makes recorded traffic stale."""
import os
import re
import shutil

import bench

CSRC = os.path.join(bench.ROOT, "long_context_layer_b200", "csrc")


def included(name, seen):
    """The local files that name includes, directly or not."""
    seen.add(name)
    for line in open(os.path.join(CSRC, name)):
        m = re.match(r'\s*#\s*include\s+"([^"]+)"', line)
        if m and m.group(1) not in seen and os.path.exists(os.path.join(CSRC, m.group(1))):
            included(m.group(1), seen)
    return seen


def test_every_source_of_the_profiled_kernels_counts(tmp_path, monkeypatch):
    d = tmp_path / "long_context_layer_b200" / "csrc"
    shutil.copytree(CSRC, d)
    before = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == before
    sources = included("delta_attn.cu", set())
    assert {"host.cuh", "launch_plain.cuh", "decode_mma.cuh"} <= sources      # the split plans and variants among them
    for name in sorted(sources):
        text = (d / name).read_text()
        (d / name).write_text(text + "\n")
        assert bench.kernel_source_hash() != before, name
        (d / name).write_text(text)
    (d / "rope.cu").write_text("other")             # other operators' sources do not
    assert bench.kernel_source_hash() == before
