"""What the host keeps per kernel holds when two threads make first calls at once (no GPU: the
runtime's calls are fakes)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def _run(tmp_path, name):
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = str(tmp_path / name)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-x", "c++", os.path.join(HERE, "host", name + ".cpp"),
                    "-I", os.path.join(ROOT, "fac_whitening_gb300", "csrc"), "-I", cuda, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_two_first_calls_of_one_kernel_keep_the_larger_limit(tmp_path):
    _run(tmp_path, "kernel_attrs_test")


def test_the_resident_ctas_are_those_of_the_launch_asked_about(tmp_path):
    _run(tmp_path, "resident_test")
