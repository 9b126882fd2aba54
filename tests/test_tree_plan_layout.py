"""Host check of the tree attention's plans (no GPU needed): tests/native/
tree_plan_check.cu evaluates the library's own planning for every accepted codec,
type and row count, and for one that cannot fit."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "native", "tree_plan_check.cu")


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return exe if os.path.exists(exe) else None


@pytest.mark.skipif(_nvcc() is None, reason="nvcc not available")
def test_tree_plans(tmp_path):
    exe = tmp_path / "tree_plan_check"
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "--expt-relaxed-constexpr",
           "-I", os.path.join(ROOT, "turboquant_kv_cache_rht_b200", "csrc"), "-I", os.path.join(ROOT, "include"),
           SRC, "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout[-4000:]
    assert "total bad 0" in run.stdout
