"""Builds the CUDA library ``libflp.so`` in-tree with nvcc for sm_103a.

The library holds the C ABI of ``include/flp.h`` and the kernels: the fused head
in ``csrc/`` and the operators beside it in ``csrc_step/``.  Their ``.cu`` files
are the translation units, compiled at the same time.  Rebuilt when any source,
or this file, is newer than the shared object.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libflp.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"
# What the generated code depends on beside the sources.  No --split-compile: it
# optimises the kernels in as many parts as it is told (0: one per CPU), and most
# kernels then come out with other registers and spills, by the machine that
# builds; the head's dX + dW launch took 5.04 ms instead of 4.79.
FLAGS = [ARCH, "-O3", "-lineinfo", "-std=c++17"]


def sources() -> list[str]:
    return (sorted(glob.glob(os.path.join(PKG, "csrc", "*")) + glob.glob(os.path.join(PKG, "csrc_step", "*")))
            + [os.path.join(ROOT, "include", "flp.h"), os.path.join(PKG, "build.py")])


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libflp.so")
    return cand


def command(out: str, extra: list[str] | None = None) -> list[str]:
    units = [s for s in sources() if s.endswith(".cu")]
    return [nvcc_path(), *FLAGS, f"--threads={len(units)}", "-Xcompiler", "-fPIC", "-shared",
            "-I" + os.path.join(ROOT, "include"), "-o", out, *units] + (extra or [])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale():
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = command(tmp, ["-Xptxas", "-v"] if verbose else None)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
