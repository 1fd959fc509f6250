"""The buffers that sherry_reserve sets aside, over a fake allocator (tests/reserve_check.cpp), and what
the library does with them."""
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sparse_bit_matmul_b200", "csrc")


def test_grown_buffers_are_kept_and_cleared(tmp_path):
    exe = tmp_path / "reserve_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "reserve_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout.startswith("ok"), res.stdout + res.stderr


def test_the_reset_clears_through_them():
    """sherry_last_device_status clears all of a device's split-K buffers, not the newest alone."""
    text = open(os.path.join(CSRC, "sherry_cuda.cu")).read()
    body = text[text.index("int sherry_last_device_status"):]
    assert re.search(r"clear_reserved\(\s*g_ws\[dev\],", body)
    assert "cudaMemset(g_ws" not in text
