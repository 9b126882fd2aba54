"""The host's check that the tree attention's shared memory starts where its plans
assume (a GPU's attributes are read, nothing is launched)."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "native", "smem_base_check.cu")
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"


@pytest.mark.skipif(not os.path.exists(NVCC), reason="nvcc not available")
def test_a_kernel_placed_elsewhere_is_refused(tmp_path):
    exe = tmp_path / "smem_base_check"
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "--expt-relaxed-constexpr",
           "-I", os.path.join(ROOT, "turboquant_kv_cache_rht_b200", "csrc"), "-I", os.path.join(ROOT, "include"),
           SRC, "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and "guard ok" in run.stdout, run.stdout[-2000:]
