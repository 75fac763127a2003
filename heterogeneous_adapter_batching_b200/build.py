"""Build liblora.so (the CUDA library behind include/lora.h) for sm_100a, in-tree."""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblora.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]

# Kernels whose launches count on an exact number of registers a thread: prompt_kernel hands the registers that its block was
# launched with from one warpgroup to the others, and a thread that asks for more than there are waits for good.
EXACT_REGISTERS = {"lora_prompt.cu": ("prompt_kernel", 168)}


def check_registers(log: str, kernel: str, count: int) -> int:
    """Instances of `kernel` in the output of `ptxas -v`; RuntimeError if one has another number of registers, or there is none."""
    found = re.findall(r"Compiling entry function '(\S*%s\S*)'.*?Used (\d+) registers" % kernel, log, re.S)
    wrong = [(name, int(n)) for name, n in found if int(n) != count]
    if wrong or not found:
        raise RuntimeError(f"{kernel} needs {count} registers a thread: {wrong or 'not found in the output of ptxas -v'}")
    return len(found)


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not _stale():
        return LIB
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        need = EXACT_REGISTERS.get(os.path.basename(src))
        if need:
            done = subprocess.run([*cmd, "-Xptxas", "-v"], stderr=subprocess.PIPE, text=True)
            if verbose or done.returncode:
                print(done.stderr, file=sys.stderr)
            done.check_returncode()
            check_registers(done.stderr, *need)
        else:
            subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
