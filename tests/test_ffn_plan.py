"""The feed-forward launches' plans, checked on the host: tile choice and work
split of the tensor-core kernel (tests/ffn_plan_check.cu), and the decode
kernel's work split and indexing (tests/ffn_decode_plan_check.cu)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.mark.skipif(not (os.path.exists(NVCC) or shutil.which("nvcc")), reason="nvcc not available")
@pytest.mark.parametrize("name", ["ffn_plan_check", "ffn_decode_plan_check"])
def test_plan_covers_and_fits(tmp_path, name):
    exe = tmp_path / name
    nvcc = NVCC if os.path.exists(NVCC) else shutil.which("nvcc")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "sparse_bit_matmul_b200", "csrc"),
                    os.path.join(HERE, name + ".cu"), "-o", str(exe)], check=True,
                   capture_output=True, text=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.startswith("ok")
