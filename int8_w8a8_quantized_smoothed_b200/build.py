"""Builds the sm_100a shared library ``libw8a8.so`` in-tree with nvcc.

    python -m int8_w8a8_quantized_smoothed_b200.build [--force] [--verbose]

The C ABI is declared in ``include/w8a8.h`` at the repository root. The runtime is linked
statically, so the library depends only on the NVIDIA driver at run time.
"""
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libw8a8.so")
SOURCES = [os.path.join(CSRC, f) for f in ("w8a8.cu", "grad.cu")]
OBJ_DIR = os.path.join(PKG, "_build")
DEPS = SOURCES + sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")) + [
    os.path.join(ROOT, "include", "w8a8.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def deps(src: str):
    """The source file and the headers it includes, directly or through another header."""
    found, todo = set(), [src]
    while todo:
        path = todo.pop()
        if path in found:
            continue
        found.add(path)
        with open(path) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                todo += [p for p in (os.path.join(CSRC, name), os.path.join(ROOT, "include", name))
                         if os.path.exists(p)]
    return sorted(found)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if it is missing or older than any source file."""
    if not force and os.path.exists(LIB):
        lib_t = os.path.getmtime(LIB)
        if all(os.path.getmtime(d) <= lib_t for d in DEPS):
            return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    jobs, objs = [], []
    for src in SOURCES:  # one compiler per source, side by side
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        objs.append(obj)
        if not force and os.path.exists(obj) and all(
                os.path.getmtime(d) <= os.path.getmtime(obj) for d in deps(src)):
            continue
        cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        # an object takes its place only when it is whole: one cut short would count as built
        cmd += ["-c", src, "-o", f"{obj}.{os.getpid()}.tmp.o"]
        jobs.append((cmd, obj, subprocess.Popen(cmd)))
    failed = []
    for cmd, obj, p in jobs:
        if p.wait() != 0:
            failed.append(cmd)
        else:
            os.replace(cmd[-1], obj)
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    subprocess.run([nvcc(), *LINK_FLAGS, *objs, "-o", LIB + ".tmp"], check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
