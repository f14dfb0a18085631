"""The recorded DRAM traffic of the bench's kernels goes with their sources,
and only with theirs."""

import os
import re
import shutil

import bench

CSRC = os.path.join(bench.ROOT, "partition_pass_tile_gb300", "csrc")
KERNELS = ("scan.cu", "select.cu", "partition.cu", "shard.cu", "api.cu")


def sources_of(names):
    """The files and what they include, directly or not."""
    found, todo = set(), list(names)
    while todo:
        name = todo.pop()
        if name in found:
            continue
        found.add(name)
        with open(os.path.join(CSRC, name)) as f:
            todo += [h for h in re.findall(r'#include "([^"/]+)"', f.read())]
    return found


def test_the_hash_covers_the_kernels_and_what_they_include():
    assert set(os.listdir(CSRC)) - bench.TRAFFIC_SOURCES_EXCLUDED == sources_of(KERNELS)


def test_other_sources_leave_the_record_valid(tmp_path, monkeypatch):
    # with the record made for the present kernels: a change elsewhere keeps it, a change of theirs does not
    shutil.copytree(CSRC, tmp_path / "partition_pass_tile_gb300" / "csrc")
    (tmp_path / "profiles").mkdir()
    (tmp_path / "profiles" / "dram_traffic.json").write_text(
        '{"split_kernel": {"n": 1024, "dram_bytes_per_launch": 16000, "source_hash": "%s"}}' % bench.kernel_source_hash())
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.recorded_traffic("split_kernel", 2048) == 32000.0
    for name in ("experts.cu", "embedding.cu", "sample.cu", "gc_rows.cuh", "radix.cu"):
        path = tmp_path / "partition_pass_tile_gb300" / "csrc" / name
        path.write_text(path.read_text() + "// more\n")
    assert bench.recorded_traffic("split_kernel", 2048) == 32000.0
    path = tmp_path / "partition_pass_tile_gb300" / "csrc" / "gc_tiles.cuh"
    path.write_text(path.read_text() + "// more\n")
    assert bench.recorded_traffic("split_kernel", 2048) is None
