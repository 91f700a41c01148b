"""Build libmsa.so in-tree with nvcc for sm_100a (B200).

    python -m top_document_sparse_b200.build [--force] [--verbose]

The library is two translation units compiled side by side (csrc/msa.cu, csrc/serve.cu; each
includes the kernel headers it needs), linked against the static CUDA runtime; it calls no driver
API directly except cuTensorMapEncodeTiled, fetched at run time through cudaGetDriverEntryPoint.
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmsa.so")
OBJ = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "msa.h")])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def _object_stale(obj: str) -> bool:
    """Whether an object is older than a file its compilation read (nvcc's -MD list)."""
    dep = obj[:-2] + ".d"
    if not (os.path.exists(obj) and os.path.exists(dep)):
        return True
    t = os.path.getmtime(obj)
    names = open(dep).read().split(":", 1)[1].replace("\\\n", " ").split()
    return any(not os.path.exists(n) or os.path.getmtime(n) > t for n in names)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    tag = f".tmp{os.getpid()}"
    objs, jobs = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if not force and not _object_stale(obj):
            continue
        cmd = [NVCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-MD", "-MF",
               obj[:-2] + ".d" + tag, "-c", src, "-o", obj + tag]
        if verbose:
            cmd[1:1] = ["-Xptxas", "-v"]
            print(" ".join(cmd), file=sys.stderr)
        jobs.append((obj, cmd, subprocess.Popen(cmd)))
    codes = [p.wait() for _, _, p in jobs]
    for (obj, cmd, _), code in zip(jobs, codes):
        if code != 0:
            raise subprocess.CalledProcessError(code, cmd)
        os.replace(obj[:-2] + ".d" + tag, obj[:-2] + ".d")
        os.replace(obj + tag, obj)
    subprocess.check_call([NVCC, *FLAGS, "-shared", *objs, "-o", LIB + tag])
    os.replace(LIB + tag, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
