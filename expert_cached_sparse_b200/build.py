"""Builds libmoe.so (all CUDA sources under csrc/) in-tree for sm_100a with nvcc."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe.so")
BUILD = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills,-v"]
# Kernels that move registers between their warps (setmaxnreg), by source and mangled name: they start
# only with the number of registers their source counts on (kRegs), and refuse to run with another.
MOVE_REGISTERS = {
    "grouped_gemm.cu": [r"gg_kernelILi2ELi256ELi1ELb0E", r"gg_kernelILi0ELi256ELi2ELb1E", r"gg_kernelILi1ELi256ELi2ELb1E"],
    "grouped_gemm_fp8.cu": [r"gg8_kernelINS0_3CfgILb0E"],
}


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(os.path.dirname(HERE), "include", "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _kernels(ptxas: str) -> dict:
    """Registers of each kernel in what ptxas -v prints."""
    return {m[1]: int(m[2]) for m in re.finditer(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", ptxas, re.S)}


def check_registers(source: str, text: str, ptxas: str) -> None:
    """Raises unless the kernels of `source` (its name and text) that move registers have kRegs of them."""
    used = _kernels(ptxas)
    for pattern in MOVE_REGISTERS.get(source, []):
        want = int(re.search(r"\bkRegs = (\d+)", text)[1])
        got = [n for k, n in used.items() if re.search(pattern, k)]
        if got != [want]:
            raise RuntimeError(f"{source}: {pattern} must be compiled to {want} registers, once; ptxas says {got}")


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs, hdrs = _sources(), _headers()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    jobs = [(s, o) for s, o in zip(srcs, objs) if force or _stale(o, [s] + hdrs)]

    def compile_one(so):
        s, o = so
        cmd = [NVCC, *ARCH, *FLAGS, "-c", s, "-o", o + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            raise RuntimeError(f"nvcc failed on {os.path.basename(s)}:\n{r.stderr}")
        with open(s) as f:
            check_registers(os.path.basename(s), f.read(), r.stderr)
        os.replace(o + ".tmp", o)
        return "\n".join(line for line in r.stderr.splitlines() if "warning" in line)

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        for msg in ex.map(compile_one, jobs):
            if verbose and msg:
                print(msg)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcuda"]
        subprocess.run(cmd, check=True, capture_output=True, text=True)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
