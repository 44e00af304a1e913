"""Builds libpa.so (CUDA kernels + C ABI + host block manager) in-tree for sm_100a."""
from __future__ import annotations

import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpa.so")

CUDA_SOURCES = ["api.cu", "append.cu", "decode_simt.cu", "decode_tensor.cu", "decode_stream.cu", "merge.cu", "decode_noalloc.cu", "rope.cu", "prefill.cu", "prefill_tc.cu", "prefill_ws.cu", "append_e2m1.cu", "decode_e2m1.cu", "prefill_wide.cu"]
CXX_SOURCES = ["block_manager.cpp", "block_pool.cpp"]
HEADERS = ["pa_internal.h", "pa_device.cuh", "pa_ptx.cuh", "pa_umma.cuh", "pa_e2m1.cuh"]

NVCC_FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Xptxas", "-v"]

# Kernels that move registers between their warps (setmaxnreg), whose shares add up to this launch number: the
# launch refuses another, so a build that came out with one is no build.
LAUNCH_REGISTERS = {"prefill_wide.cu": ("prefill_wide_kernel", 128)}


def check_registers(ptxas: str, kernel: str, want: int) -> int:
    """Number of `kernel`'s instantiations in ptxas' report; raises if one has not `want` registers."""
    entries = re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", ptxas, re.S)
    got = [int(n) for name, n in entries if kernel in name]
    if not got or any(n != want for n in got):
        raise RuntimeError("%s: %s registers a thread, its warps' shares are for %d" % (kernel, got or "no", want))
    return len(got)


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    common = [os.path.join(INCLUDE, "pa.h")] + [os.path.join(CSRC, h) for h in HEADERS]
    objs = []
    for src in CUDA_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + common):
            cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", s, "-o", o]
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                sys.stderr.write(res.stdout + res.stderr)
                raise RuntimeError("nvcc failed on %s" % src)
            if src in LAUNCH_REGISTERS:
                try:
                    check_registers(res.stderr, *LAUNCH_REGISTERS[src])
                except RuntimeError:
                    os.remove(o)               # the next build compiles it again
                    raise
            with open(o + ".ptxas.txt", "w") as f:
                f.write(res.stderr)
            if verbose:
                sys.stderr.write(res.stderr)
    for src in CXX_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + common):
            subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                                   "-I", INCLUDE, "-I", CSRC, "-c", s, "-o", o])
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        subprocess.check_call([_nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
                               *objs, "-o", tmp, "-cudart", "static"])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
