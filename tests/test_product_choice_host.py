"""The choice of a product's launch (mhcm_product.cu) keeps every access to shared
memory inside what it asks for, over many shapes (host code, no GPU needed)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "rms_backward_gb300", "csrc")


def _cuda_include():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")


def test_shared_memory_holds_what_is_touched(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(_cuda_include(), "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = tmp_path / "choice"
    build = subprocess.run(["g++", "-std=c++17", "-O2", "-I", _cuda_include(), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                            "-x", "c++", os.path.join(CSRC, "mhcm_product.cu"), os.path.join(HERE, "c", "product_choice.cpp"),
                            "-o", str(exe)], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout
