"""Build libbfmoe.so in-tree with nvcc for sm_100a.

    python -m ternary_butterfly_experts_b200.build [-v]

The library links the CUDA runtime statically, so it loads next to any
PyTorch build; the driver's tensor-map encoder is looked up at run time.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbfmoe.so")
OBJ = os.path.join(PKG, "_build")   # one object per translation unit

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return [os.path.join(CSRC, "bfmoe.cu"), os.path.join(CSRC, "route.cu")]


def deps(source=None):
    """The header and kernel files that the library (or one source) is built from."""
    todo, seen = [source] if source else sources(), []
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.append(path)
        with open(path) as f:
            names = re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M)
        for n in names:
            todo += [q for q in (os.path.join(CSRC, n), os.path.join(INCLUDE, n)) if os.path.exists(q)]
    return sorted(seen)


def newer(target, paths) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in paths)


def up_to_date() -> bool:
    return newer(LIB, deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    common = [nvcc(), *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if ptxas_info:
        common.insert(1, "-Xptxas=-v")

    def start(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)

    def finish(what, p):
        out = p.communicate()[0]
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {what} ({p.returncode}):\n{out}")
        if verbose or ptxas_info:
            sys.stdout.write(out)

    mine = f".{os.getpid()}.tmp"   # two builds at once do not meet
    objects, running = [], []
    for src in sources():
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objects.append(obj)
        if force or not newer(obj, deps(src)):
            running.append((src, obj, start([*common, "-c", src, "-o", obj + mine])))
    failed = None
    for src, obj, p in running:   # every compiler is waited for, also after a failure
        try:
            finish(src, p)
            os.replace(obj + mine, obj)
        except RuntimeError as e:
            failed = failed or e
    if failed:
        raise failed
    finish(LIB, start([nvcc(), *ARCH, "--shared", "-Xcompiler", "-fPIC", "-cudart", "static", *objects,
                       "-o", LIB + mine, "-ldl", "-lpthread", "-lrt"]))
    os.replace(LIB + mine, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
