"""Build ``libcce.so`` (the C-ABI library) in-tree for sm_100a with nvcc.

    python -m lm_head_cross_flash_b200.build [--force]

The library is rebuilt when any source under ``csrc/`` or ``include/`` is
newer than it.  No GPU is needed: nvcc cross-compiles for sm_100a.
"""

from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libcce.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-v",
]


def _nvcc() -> str:
    for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(SRC, "*.cu")) + glob.glob(os.path.join(SRC, "*.cuh"))
                  + glob.glob(os.path.join(ROOT, "include", "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


# Kernels that hand registers from some warps to others (setmaxnreg): the sum
# is counted against this many a thread at launch, and the library refuses to
# run such a kernel when it was compiled to another number.
REGISTERS = {"fp8_rows_kernel": 168}


def check_registers(ptxas_log: str) -> None:
    """Raise RuntimeError unless ptxas -v reports REGISTERS."""
    for kernel, want in REGISTERS.items():
        got = re.findall(r"entry function '\w*" + kernel + r"\w*'(?:.*\n)+?.*Used (\d+) registers",
                         ptxas_log)
        if [int(n) for n in got] != [want]:
            raise RuntimeError(f"{kernel}: compiled to {got} registers, its hand-over needs {want}")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"),
           "-o", LIB + ".tmp", os.path.join(SRC, "cce.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    log = os.path.join(PKG, "build.log")
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stderr[-4000:]}")
    check_registers(r.stdout + r.stderr)
    os.replace(LIB + ".tmp", LIB)
    if verbose:
        print(r.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
