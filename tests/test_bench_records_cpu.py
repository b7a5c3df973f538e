"""The benchmark's traffic records: those that are kept were taken from the kernels' present sources, and what the public
header declares behind the convolution's part does not concern them."""
from __future__ import annotations

import os
import shutil

import pytest

import bench
import workloads


@pytest.mark.parametrize("name", ["mamba2_inconv_headwise", "qkv_150m_lowrank"])
def test_records_count(name):
    w = workloads.WORKLOADS[name]
    measured = bench.measured_traffic("bwd_conv", w)
    assert measured is not None and measured >= bench.algorithmic_bytes(w)["bwd_conv"] * w.tokens


@pytest.mark.parametrize("kind", ["headwise", "lowrank"])
def test_what_a_record_depends_on(kind, tmp_path, monkeypatch):
    sha = bench.kernel_source_sha("bwd_conv", kind)
    for part in ("include", os.path.join("input_dependent_depthwise_amd", "csrc")):
        shutil.copytree(os.path.join(bench.ROOT, part), tmp_path / part)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    header = tmp_path / "include" / "dynconv.h"
    text = header.read_text()
    assert bench.kernel_source_sha("bwd_conv", kind) == sha
    header.write_text(text + "/* another call */\n")
    assert bench.kernel_source_sha("bwd_conv", kind) == sha
    header.write_text("/* another convolution */\n" + text)
    assert bench.kernel_source_sha("bwd_conv", kind) != sha
    header.write_text(text)
    own = tmp_path / "input_dependent_depthwise_amd" / "csrc" / bench.KERNEL_SOURCES[("bwd_conv", kind)][0]
    own.write_text(own.read_text() + "\n")
    assert bench.kernel_source_sha("bwd_conv", kind) != sha
