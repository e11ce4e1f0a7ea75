"""The routing's sigmoid takes its reciprocal from the hardware's estimate and one correction: equal to the correctly
rounded quotient for every divisor it is used for."""
import ctypes
import os
import subprocess

import pytest
import torch

from mxfp8_block_scaled_04_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def build_check(out):
    nvcc = os.path.join(CUDA, "bin", "nvcc")
    subprocess.run([nvcc if os.path.exists(nvcc) else "nvcc", build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
                    "-I", os.path.join(build.PKG, "csrc"), "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "reciprocal_check.cu"), "-o", out], check=True)


def test_reciprocal_check_compiles(tmp_path):
    build_check(str(tmp_path / "check.so"))


@pytest.mark.gpu
def test_reciprocal_is_correctly_rounded_for_every_divisor(tmp_path):
    build_check(str(tmp_path / "check.so"))
    check = ctypes.CDLL(str(tmp_path / "check.so"))
    check.reciprocal_compare.argtypes = [ctypes.c_void_p]
    out = torch.zeros(3, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    assert check.reciprocal_compare(out.data_ptr()) == 0
    compared, differ, example = out.tolist()
    assert compared == 126 * 2 ** 23 + 1  # [1, 2^126): 126 exponents, and 2^126 itself
    assert differ == 0, hex(example)
