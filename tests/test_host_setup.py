"""Host code that decides what is launched, tested without a GPU: small programs that
include the library's own headers, compiled with the host compiler."""
import glob
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp8_mixed_precision_amax_gb300", "csrc")


def run_check(name, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if not os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
        pytest.skip("no CUDA headers")
    exe = str(tmp_path / name)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I" + CSRC, "-I" + include, "-o", exe,
                    os.path.join(HERE, "host", name + ".cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_setup_runs_once_on_each_device(tmp_path):
    run_check("once_per_device_check", tmp_path)


def test_layernorm_backward_starts_what_is_resident(tmp_path):
    run_check("ln_plan_check", tmp_path)


def test_kernel_attributes_are_set_by_that_alone():
    """cudaFuncSetAttribute acts on the current device: behind a flag of the process it would
    leave the kernels of every other device without it."""
    for path in glob.glob(os.path.join(CSRC, "*")):
        if os.path.basename(path) != "once_per_device.h":
            assert "cudaFuncSetAttribute" not in open(path).read(), path
