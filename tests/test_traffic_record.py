"""bench.py reports the recorded DRAM traffic only while the GEMM's source and every header of it are those it was taken
on (no GPU)."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

CSRC = os.path.join(ROOT, "exact_modular_int8_gb300", "csrc")


@pytest.mark.parametrize("name", ["gemm_tc.cu", "rg_tc.cuh", "rg_common.cuh", "rg_kernels.h"])
def test_a_changed_source_or_header_drops_the_record(tmp_path, name):
    csrc = str(tmp_path / "csrc")
    shutil.copytree(CSRC, csrc)
    source = os.path.join(csrc, "gemm_tc.cu")
    assert bench.gemm_traffic_record(source) is not None
    with open(os.path.join(csrc, name), "a") as f:
        f.write("\n")
    assert bench.gemm_traffic_record(source) is None


def test_another_kernels_files_do_not(tmp_path):
    csrc = str(tmp_path / "csrc")
    shutil.copytree(CSRC, csrc)
    for name in ("f8_gemm.cu", "f8_kernels.h", "recon.h"):
        with open(os.path.join(csrc, name), "a") as f:
            f.write("\n")
    assert bench.gemm_traffic_record(os.path.join(csrc, "gemm_tc.cu")) is not None
