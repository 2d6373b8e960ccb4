"""Build libkvq.so in-tree for B200 (sm_100a) with nvcc.

Each CUDA source is compiled to an object under _build/ (in parallel, and
only when it or a header that it includes changed), then linked into
kv_cache_mixed_kvq_b200/libkvq.so.  Usage: python -m kv_cache_mixed_kvq_b200.build
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkvq.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--ftz=false", "--prec-div=true", "--prec-sqrt=true", "--fmad=true",
         "-I", INCLUDE, "-I", CSRC]


def _with_headers(src: str) -> set:
    """src and every header of this repository that it includes."""
    seen, todo = set(), [src]
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.add(path)
        with open(path) as f:
            names = re.findall(r'^#include "([^"]+)"', f.read(), re.M)
        todo += [p for n in names for p in (os.path.join(CSRC, n), os.path.join(INCLUDE, n))
                 if os.path.exists(p)]
    return seen


def check_launch_registers(log: str) -> None:
    """Checks the assembler's report on the chunk attention kernels: their
    warpgroups' register split counts on what the launch allocates (registers
    a thread, in eights); with less it would never be granted."""
    with open(os.path.join(CSRC, "chunk.cuh")) as f:
        want = int(re.search(r"kRegsLaunch = (\d+)", f.read()).group(1))
    kernel, seen = None, 0
    for line in log.splitlines():
        m = re.search(r"Compiling entry function '(\S+)'", line)
        if m:
            kernel = m.group(1) if "chunk_kernel" in m.group(1) else None
        m = re.search(r"Used (\d+) registers", line)
        if m and kernel:
            seen += 1
            if (int(m.group(1)) + 7) // 8 * 8 != want:
                raise RuntimeError(f"{kernel} was given {m.group(1)} registers a thread; the split "
                                   f"among its warpgroups (csrc/chunk.cuh) needs {want}")
    if not seen:
        raise RuntimeError("no report on the registers of the chunk attention kernels")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest = max(os.path.getmtime(p) for p in _with_headers(src))
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    cmd = [NVCC] + ARCH + FLAGS + ["-c", src, "-o", obj + ".tmp"]
    splits_registers = os.path.basename(src) == "chunk.cu"
    if verbose or splits_registers:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    if splits_registers:
        check_launch_registers(r.stderr)
    os.replace(obj + ".tmp", obj)
    return obj


def build(verbose: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with ThreadPoolExecutor(max_workers=jobs or os.cpu_count() or 4) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([NVCC] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
