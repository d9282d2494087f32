"""Host check (no GPU) of the barriers of the CTA-pair GEMM's ring of bits and
scales: compiles tests/native/pair_ring_check.cpp against the kernel's pair_ring.h
with the host C++ compiler and runs it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "boolean_weight_matmul_b200", "csrc")
SRC = os.path.join(ROOT, "tests", "native", "pair_ring_check.cpp")


def test_waits_for_bits_pass_behind_their_copies_only(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "pair_ring_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, SRC, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
