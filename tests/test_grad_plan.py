"""Launch shapes of the feed-forward gradients' column sums (tests/grad_plan_check.cu)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.mark.skipif(not (os.path.exists(NVCC) or shutil.which("nvcc")), reason="nvcc not available")
def test_chains_of_the_column_sums_are_short(tmp_path):
    exe = tmp_path / "grad_plan_check"
    nvcc = NVCC if os.path.exists(NVCC) else shutil.which("nvcc")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", os.path.join(os.path.dirname(HERE), "sparse_bit_matmul_b200", "csrc"),
                    os.path.join(HERE, "grad_plan_check.cu"), "-o", str(exe)], check=True, capture_output=True, text=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and res.stdout.startswith("ok"), res.stdout + res.stderr
