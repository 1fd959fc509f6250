"""The calls of ffn_cases.py take the paths they are there for, and together all that there are."""
import os
import shutil
import subprocess

import pytest

from ffn_cases import ACTS, COLUMNS, DTYPES, FORWARD, GRADIENT

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.mark.skipif(not (os.path.exists(NVCC) or shutil.which("nvcc")), reason="nvcc not available")
def test_cases_take_their_paths(tmp_path):
    exe = tmp_path / "ffn_path_query"
    nvcc = NVCC if os.path.exists(NVCC) else shutil.which("nvcc")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "sparse_bit_matmul_b200", "csrc"), os.path.join(HERE, "ffn_path_query.cu"),
                    "-o", str(exe)], check=True, capture_output=True, text=True)
    cases = list(FORWARD) + list(GRADIENT)
    args = []
    for _, kind, dt, act, _, residual, keep, M, N, K in cases:
        args += [kind, DTYPES.index(dt), ACTS.index(act), int(residual), int(keep), M, N, K]
    out = subprocess.run([str(exe)] + [str(a) for a in args], check=True, capture_output=True, text=True).stdout.split()
    assert len(out) == len(cases)
    wrong = [(case, got) for case, got in zip(cases, out) if case[0] != got]
    assert not wrong, wrong
    tiles = [f"{bn}/1/{how}" for bn in (64, 128, 192) for how in ("leftover", "splitS", "whole+")]
    tiles += [f"{bn}/1/{how}" for bn in (16, 32) for how in ("c2", "c4", "leftover", "splitS")]
    for kind in ("linear", "gated"):
        got = {c[0] for c in FORWARD if c[1] == kind}
        missing = [t for t in tiles + ["decode/2", "decode/4"] if t not in got]
        assert not missing, (kind, missing)
    for digits in (("f32",), ("bf16", "f16")):
        got = {c[0] for c in GRADIENT if c[2] in digits}
        assert {"192/2/whole+", "192/1/whole+", "192/1/leftover", "192/1/splitS", "128/1/leftover", "128/1/splitS",
                "64/1/splitS", "32/1/leftover", "16/1/splitS", "16/1/leftover", "32/1/c2", "16/1/c2"} <= got
    assert all(M > 1024 and N > 2304 for M, N, _ in COLUMNS)
