"""The shared-memory limit of a kernel, raised by two threads at once (CPU; tests/c/smem_limit_check.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_the_largest_limit_stands(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    exe = str(tmp_path / "smem_limit_check")
    cc = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I" + cuda,
                         "-I" + os.path.join(ROOT, "bit_quantized_b200", "csrc"),
                         os.path.join(ROOT, "tests", "c", "smem_limit_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
