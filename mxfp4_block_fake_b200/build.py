"""Build libmxfp4.so in-tree with nvcc for sm_100a (B200).

    python -m mxfp4_block_fake_b200.build [--force] [--verbose-ptxas]

The library is plain CUDA runtime C++ behind the C ABI of include/mxfp4.h; it
does not link against torch. The .so lands next to this file so that it
travels with the source tree.
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SRCS = ("mxfp4.cu", "mxfp4_moe.cu")  # translation units, compiled side by side
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmxfp4.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def _sources(path: str, seen: set | None = None) -> set:
    """path and every file of this tree it includes."""
    seen = set() if seen is None else seen
    if path not in seen:
        seen.add(path)
        with open(path) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                for d in (CSRC, INCLUDE):
                    if os.path.exists(os.path.join(d, name)):
                        _sources(os.path.join(d, name), seen)
    return seen


def _stale(out: str, deps) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(p) > os.path.getmtime(out) for p in deps)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    deps = {s: _sources(os.path.join(CSRC, s)) | {os.path.abspath(__file__)} for s in SRCS}
    if not force and not verbose_ptxas and not _stale(LIB, set().union(*deps.values())):
        return LIB
    os.makedirs(OBJ, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ, src + ".o")
        if force or verbose_ptxas or _stale(obj, deps[src]):
            cmd = [NVCC, *NVCC_FLAGS, "-I", INCLUDE, "-c", "-o", obj + ".tmp", os.path.join(CSRC, src)]
            if verbose_ptxas:
                cmd[1:1] = ["-Xptxas", "-v"]
            subprocess.run(cmd, check=True)
            os.replace(obj + ".tmp", obj)
        return obj

    with ThreadPoolExecutor(len(SRCS)) as pool:
        objs = list(pool.map(compile_one, SRCS))
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", LIB + ".tmp", *objs], check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv))
