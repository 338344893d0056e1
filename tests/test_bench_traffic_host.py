"""The bench reports DRAM traffic while the measured kernels are the current
ones, and only then: changes to kernels that its steps do not launch do not
count, changes to theirs do."""
import json
import os
import shutil

import pytest

import bench
from gemm_epilogues_tcgen05_b200 import synth


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the kernel sources and the traffic file, at the current hash."""
    csrc = tmp_path / "gemm_epilogues_tcgen05_b200" / "csrc"
    shutil.copytree(os.path.join(bench.ROOT, "gemm_epilogues_tcgen05_b200", "csrc"), csrc)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    (tmp_path / "profiles").mkdir()
    entry = {"dram_bytes_per_launch": 1234, "source_hash": bench.kernel_source_hash()}
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps({"ffn:bwd": entry}))
    return csrc


def measured():
    return bench.measured_traffic(synth.WORKLOADS["ffn"], "bwd", "RELU_AUX_BIAS")


def append(path):
    path.write_text(path.read_text() + "\n// another line\n")


@pytest.mark.parametrize("unit", ["grouped_kernel.cuh", "grouped.cu", "mx.cu", "mx_quant.cuh", "mx_kernel.cuh", "inst_mx.cu",
                                  "inst_grouped.cuh"])
def test_kernels_beside_the_measured_ones_keep_the_evidence(tree, unit):
    every = bench.kernel_source_hash(every_unit=True)
    append(tree / unit)
    assert measured() == 1234 and bench.kernel_source_hash(every_unit=True) != every


@pytest.mark.parametrize("unit", ["tile2_kernel.cuh", "tile_kernel.cuh", "skinny_kernel.cuh", "aux_kernels.cuh", "ptx.cuh",
                                  "gemm_epi.cu", "host_common.h", "inst_pair_bf16.cu"])
def test_the_measured_kernels_void_it(tree, unit):
    append(tree / unit)
    assert measured() is None


def test_every_committed_entry_names_one_hash():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        entries = [v for v in json.load(f).values() if isinstance(v, dict)]
    assert len({v["source_hash"] for v in entries}) == 1 and all(v["dram_bytes_per_launch"] > 0 for v in entries)
