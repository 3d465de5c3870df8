"""The recorded DRAM traffic of the headline's kernel stands as long as that kernel does (no GPU)."""
from __future__ import annotations

import os
import re

import bench


def _included_by(name):
    """The csrc files that `name` includes, directly or through others, and itself."""
    found, left = set(), [name]
    while left:
        n = left.pop()
        if n in found or not os.path.exists(os.path.join(bench.DOMINANT_KERNEL_SRC, n)):
            continue
        found.add(n)
        with open(os.path.join(bench.DOMINANT_KERNEL_SRC, n), encoding="utf-8") as f:
            left += re.findall(r'^#include "([^"]+)"', f.read(), re.M)
    return found


def test_other_kernels_sources_hold_none_of_the_partials_kernel():
    kernel = _included_by("partials_tc.cu")
    assert {"partials_tc.cu", "ls_plan.cuh", "ls_device.cuh", "sm100.cuh"} <= kernel
    assert not kernel & set(bench.OTHER_KERNELS)
    assert set(bench.OTHER_KERNELS) <= set(os.listdir(bench.DOMINANT_KERNEL_SRC))


def test_a_new_kernels_file_leaves_the_record_alone(monkeypatch, tmp_path):
    (tmp_path / "partials_tc.cu").write_text("int a;\n")
    (tmp_path / "sample.cu").write_text("int b;\n")
    monkeypatch.setattr(bench, "DOMINANT_KERNEL_SRC", str(tmp_path))
    before = bench.kernel_source_hash()
    (tmp_path / "sample.cu").write_text("int c;\n")
    assert bench.kernel_source_hash() == before
    (tmp_path / "partials_tc.cu").write_text("int d;\n")
    assert bench.kernel_source_hash() != before


def test_the_headline_has_its_traffic():
    """Fails once the kernel's own sources changed: capture it again and record it in
    profiles/traffic.json, with bench.kernel_source_hash()."""
    assert bench.recorded_traffic(bench.HEADLINE.name) is not None


def test_another_plan_has_no_record():
    plan = {"partials_ctas": 144, "blocks_per_chunk": 29, "combine_ctas": 448}
    assert bench.recorded_traffic(bench.HEADLINE.name, plan) is not None
    assert bench.recorded_traffic(bench.HEADLINE.name, {**plan, "blocks_per_chunk": 30}) is None
