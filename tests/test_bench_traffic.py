"""The committed HBM counter summaries belong to the kernels as they are now, so that bench.py
reports them, and are tied to what those kernels are built from and to nothing else."""
import json
import os
import re

import pytest

import bench

ROOT = bench.ROOT
CSRC = os.path.join(ROOT, "selective_state_space_vjp_amd", "csrc")
SUMMARIES = ["ssd_chunk16_kernel", "ssd_state_scan_kernel", "ssd_blocked_bwd_kernel"]


@pytest.mark.parametrize("kernel", SUMMARIES)
def test_counter_summary_is_of_the_present_sources(kernel):
    rec = json.load(open(os.path.join(ROOT, "profiles", f"traffic_{kernel}.json")))
    assert rec["kernel"] == kernel and rec["sources"] == list(bench.KERNEL_SOURCES[kernel])
    assert bench.traffic_from_profile(kernel) == rec["bytes_per_launch"]
    # what the counters read is what the kernel has to move, and not twice that
    assert 1.0 <= rec["bytes_per_launch"] / rec["algorithmic_bytes"] < 1.5


@pytest.mark.parametrize("kernel", bench.KERNEL_SOURCES)
def test_sources_are_the_file_and_the_headers_it_includes(kernel):
    first = os.path.basename(bench.KERNEL_SOURCES[kernel][0])
    seen, todo = {first}, [first]
    while todo:
        text = open(os.path.join(CSRC, todo.pop())).read()
        new = set(re.findall(r'#include "(\w+\.cuh)"', text)) - seen
        seen |= new
        todo += new
    assert {os.path.basename(f) for f in bench.KERNEL_SOURCES[kernel]} == seen


def test_other_files_of_the_library_do_not_matter(monkeypatch):
    from selective_state_space_vjp_amd import _build

    before = {k: bench.sources_sha256(k) for k in bench.KERNEL_SOURCES}
    monkeypatch.setattr(_build, "SOURCES", _build.SOURCES + ["another.hip"])
    monkeypatch.setattr(_build, "EXTRA", dict(_build.EXTRA, **{"another.hip": ["-O1"]}))
    assert {k: bench.sources_sha256(k) for k in bench.KERNEL_SOURCES} == before
    monkeypatch.setattr(_build, "EXTRA", {})
    changed = {k for k in before if bench.sources_sha256(k) != before[k]}
    assert changed == {"ssd_chunk16_kernel"}
