"""The choice of a product's launch (mhcm_product.cu) for long sums (host code, no GPU
needed)."""
import os
import shutil
import subprocess

import pytest

from test_product_choice_host import CSRC, HERE, ROOT, _cuda_include


def test_long_sums_fit(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(_cuda_include(), "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = tmp_path / "choice"
    build = subprocess.run(["g++", "-std=c++17", "-O2", "-I", _cuda_include(), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                            "-x", "c++", os.path.join(CSRC, "mhcm_product.cu"), os.path.join(HERE, "c", "product_long_sums.cpp"),
                            "-o", str(exe)], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout
