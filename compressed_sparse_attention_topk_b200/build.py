"""Build libcsa2.so (sm_100a) in-tree with nvcc.

Usage: python -m compressed_sparse_attention_topk_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libcsa2.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

SOURCES = ["csa2.cu", "kv8.cu"]
OBJ = os.path.join(PKG, "_build")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "csa2.h"))
    return files


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _stale(obj: str, dep: str) -> bool:
    """Whether an object is older than a file that it was compiled from (the
    compiler's own dependency list; files outside the tree do not count)."""
    if not os.path.exists(obj) or not os.path.exists(dep):
        return True
    t = os.path.getmtime(obj)
    with open(dep) as f:
        words = f.read().replace("\\\n", " ").split()[1:]
    ours = [w for w in words if os.path.abspath(w).startswith(ROOT + os.sep)]
    return not ours or any(not os.path.exists(w) or os.path.getmtime(w) > t for w in ours)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
             "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if verbose:
        flags += ["-Xptxas", "-v"]
    tag = f".tmp{os.getpid()}"
    objects, running = [], []
    for s in SOURCES:
        obj = os.path.join(OBJ, os.path.splitext(s)[0] + ".o")
        dep = obj[:-2] + ".d"
        objects.append(obj)
        if force or verbose or _stale(obj, dep):
            cmd = [NVCC, *flags, "-MD", "-MF", dep + tag, "-c", "-o", obj + tag,
                   os.path.join(CSRC, s)]
            running.append((cmd, obj, dep, subprocess.Popen(cmd)))
    failed = [cmd for cmd, _, _, p in running if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, obj, dep, _ in running:
        os.replace(obj + tag, obj)
        os.replace(dep + tag, dep)
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o",
                    LIB + tag, *objects], check=True)
    os.replace(LIB + tag, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
