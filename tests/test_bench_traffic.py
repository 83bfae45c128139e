"""bench.py reports counted HBM traffic only for the kernel source that it was
counted on: the file and the device code that it includes.  No GPU."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

CSRC = os.path.join("w4a4_rank_corrected_quantize_amd", "csrc")


@pytest.fixture
def copy(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(ROOT, CSRC), str(tmp_path / CSRC))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))

    def edit(name, old, new):
        path = tmp_path / CSRC / name
        text = path.read_text()
        assert old in text
        path.write_text(text.replace(old, new, 1))
    return edit


@pytest.mark.parametrize("workload", ["fc1", "mx_fc1"])
@pytest.mark.parametrize("name,old,new", [
    ("w4a4_gemm.hip", "store_nt(", "store_all("), ("w4a4_epilogue.h", "-0.102943836f", "-0.102943837f"),
    ("svdq_quant.h", "__device__", "__device__ __noinline__")])
def test_changed_device_code_has_no_traffic(copy, workload, name, old, new):
    kept = bench.TRAFFIC[workload]["bytes"]
    assert bench.measured_traffic(workload) in (kept, None)
    before = bench._source_sha("w4a4_gemm.hip")
    copy(name, old, new)
    assert bench._source_sha("w4a4_gemm.hip") != before
    assert bench.measured_traffic(workload) is None


@pytest.mark.parametrize("name,old,new", [
    ("w4a4_epilogue.h", "// SiLU", "// The SiLU"), ("svdq_internal.h", "hipError_t launch_rope_table(", "hipError_t  launch_rope_table("),
    ("rope.hip", "float", "double")])
def test_comments_and_other_calls_do_not_count(copy, name, old, new):
    before = bench._source_sha("w4a4_gemm.hip")
    copy(name, old, new)
    assert bench._source_sha("w4a4_gemm.hip") == before
