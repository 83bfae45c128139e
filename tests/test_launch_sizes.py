"""Launch sizes against what the runtime takes, on the CPU: a small C++ program
built against the library's own header sweeps the sizes that a call accepts."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "w4a4_rank_corrected_quantize_amd", "csrc")


def _run(source, tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-I", CSRC, os.path.join(HERE, "native", source), "-o", exe],
                   check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_attention_launches(tmp_path):
    _run("kv4_plan_check.cpp", tmp_path)


def test_residual_norm_launches(tmp_path):
    _run("launch_grid_check.cpp", tmp_path)
