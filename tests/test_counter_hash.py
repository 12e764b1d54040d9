"""The hash that ties committed counters to the kernels they were taken on."""
import json

import pytest

import bench
from gated_delta_rule_55_amd import build


def test_committed_counters_belong_to_these_kernels():
    with open(bench.COUNTERS_FILE) as f:
        assert json.load(f)["source_hash"] == bench.kernel_source_hash()
    assert bench.measured_counter("prefill", "bytes_per_launch") > 0


def test_other_sources_and_steps_of_the_build_do_not_retire_counters(monkeypatch):
    was = bench.kernel_source_hash()
    monkeypatch.setattr(build, "SOURCES", build.SOURCES + ["another.hip"])
    monkeypatch.setattr(build, "SOURCE_FLAGS", dict(build.SOURCE_FLAGS, **{"another.hip": ["-O1"]}))
    monkeypatch.setattr(build, "HIPCC_FLAGS", build.HIPCC_FLAGS + ["-I/elsewhere"])
    assert bench.kernel_source_hash() == was


@pytest.mark.parametrize("what", ["flags", "source flags", "arch", "source"])
def test_what_shapes_the_kernels_does(monkeypatch, tmp_path, what):
    was = bench.kernel_source_hash()
    if what == "flags":
        monkeypatch.setattr(build, "HIPCC_FLAGS", build.HIPCC_FLAGS + ["-ffast-math"])
    elif what == "source flags":
        monkeypatch.setattr(build, "SOURCE_FLAGS", {})
    elif what == "arch":
        monkeypatch.setattr(build, "HIPCC_FLAGS", [f.replace(build.ARCH, "gfx1") for f in build.HIPCC_FLAGS])
    else:
        for rel in bench.KERNEL_SOURCES:
            (tmp_path / rel).parent.mkdir(parents=True, exist_ok=True)
            (tmp_path / rel).write_text(open(f"{bench.ROOT}/{rel}").read() + "int one_more;\n")
        monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() != was
    assert bench.measured_counter("prefill", "bytes_per_launch") is None
