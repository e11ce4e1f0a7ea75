"""Build the CUDA library ``_build/libmxfp8.so`` in-tree for sm_103a (GB300).

    python -m mxfp8_block_scaled_04_gb300.build

nvcc cross-compiles without a GPU.  No fast-math: the kernels rely on
IEEE fp32 multiplies that keep subnormals.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libmxfp8.so")
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("api.cu", "mxfp4.cu", "moe.cu")]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def _inputs():
    return (SOURCES + glob.glob(os.path.join(PKG, "csrc", "*.cuh")) + glob.glob(os.path.join(PKG, "csrc", "*.h")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    if not os.path.exists(nvcc):
        nvcc = "nvcc"
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    flags = [ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags.insert(0, "-Xptxas=-v")
    objects, running = [], []
    for src in SOURCES:  # one nvcc per translation unit, side by side
        obj = os.path.join(BUILD_DIR, f"{os.path.splitext(os.path.basename(src))[0]}.tmp{os.getpid()}.o")
        cmd = [nvcc] + flags + ["-c", "-o", obj, src]
        if verbose:
            print(" ".join(cmd), flush=True)
        objects.append(obj)
        running.append((cmd, subprocess.Popen(cmd)))
    codes = [p.wait() for _, p in running]
    try:
        for (cmd, _), code in zip(running, codes):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.run([nvcc, ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objects, check=True)
    finally:
        for obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
