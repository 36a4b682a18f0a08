"""Build libmoe.so in-tree with nvcc for sm_103a (no cmake; the translation units compile in parallel)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoe.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def nvcc_path() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    flags = [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE]
    if verbose:
        flags.insert(1, "-Xptxas=-v")
    with tempfile.TemporaryDirectory(dir=PKG, prefix="_build") as d:
        units = [(src, os.path.join(d, os.path.basename(src)[:-3] + ".o"))
                 for src in sorted(glob.glob(os.path.join(CSRC, "*.cu")))]
        jobs = [subprocess.Popen([*flags, "-c", src, "-o", obj], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                 text=True) for src, obj in units]
        logs = [j.communicate()[0] for j in jobs]
        if any(j.returncode for j in jobs):
            sys.stderr.write("".join(logs))
            raise RuntimeError("nvcc failed building libmoe.so")
        r = subprocess.run([nvcc_path(), *ARCH, "-shared", *[obj for _, obj in units], "-o", tmp],
                           capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc failed linking libmoe.so")
    if verbose:
        sys.stderr.write("".join(logs))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
