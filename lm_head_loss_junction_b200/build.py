"""Builds libmls.so in-tree with nvcc for sm_100a.

    python -m lm_head_loss_junction_b200.build

The library links the CUDA runtime statically and reaches the driver API
(cuTensorMapEncodeTiled) at run time, so it loads on machines without a GPU.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmls.so")
SOURCES = ["api.cu", "junction.cu", "segsum.cu", "loss_simt.cu", "loss_tc.cu", "junction_noalloc.cu",
           "head_api.cu", "head_tc.cu", "head_few.cu", "head_rows.cu", "head_simt.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


HASH = LIB + ".srchash"


def source_hash() -> str:
    """SHA-256 over every source file, the public header and the compiler flags.

    Content, not modification times: a copied tree (whose files all get new
    times) keeps a valid library, and an edited source always rebuilds it.
    """
    h = hashlib.sha256()
    deps = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)) + [os.path.join(INCLUDE, "mls.h")]
    for d in deps:
        h.update(os.path.basename(d).encode())
        with open(d, "rb") as f:
            h.update(f.read())
    h.update(" ".join(ARCH + SOURCES).encode())
    return h.hexdigest()


def _stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(HASH)):
        return True
    with open(HASH) as f:
        return f.read().strip() != source_hash()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles libmls.so unless the library on disk was built from the current sources."""
    if not force and not _stale():
        return LIB
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    common = [nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        common += ["-Xptxas", "-v"]
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.run([nvcc(), *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    with open(HASH, "w") as f:
        f.write(source_hash() + "\n")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
