"""A device's set-up that fails is tried again by the next call: the operators'
host code, compiled as plain C++ against a stand-in for the CUDA runtime
(tests/c/operators_setup_fails_once.cpp)."""
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


def test_a_failed_setup_is_not_kept(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(_cuda_include(), "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = tmp_path / "setup"
    build = subprocess.run(["g++", "-std=c++17", "-I", _cuda_include(), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                            "-x", "c++", os.path.join(CSRC, "mhcs_api.cu"),
                            os.path.join(HERE, "c", "operators_setup_fails_once.cpp"), "-pthread", "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    run = subprocess.run([str(exe)], timeout=60)
    assert run.returncode == 0, f"operators_setup_fails_once.cpp:{run.returncode}"
