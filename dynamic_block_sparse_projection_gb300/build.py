"""Build libdsv.so (the C-ABI library) for sm_103a with nvcc, in-tree.

One nvcc process per translation unit, run in parallel, then one link step.
Output: dynamic_block_sparse_projection_gb300/_build/libdsv.so, and beside it the
CPython module dsv_calls, linked against it.  The module's file name carries the
interpreter's version and machine, so that one built for another interpreter is
neither loaded nor taken for this one's.  Rebuilds only when a source or header
is newer than the outputs.
"""
from __future__ import annotations

import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
OUT = PKG / "_build"
LIB = OUT / "libdsv.so"
CALLS = OUT / ("dsv_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])
SOURCES = ["dsv_api.cu", "predict.cu", "topk.cu", "attn_fwd.cu", "attn_bwd.cu", "topk_noalloc.cu", "cube.cu",
           "predict_max.cu", "predict_topk.cu", "packed_fwd.cu", "packed_bwd.cu", "rope.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdsv")


def _inputs():
    return [CSRC / s for s in SOURCES + ["pycalls.c"]] + list(CSRC.glob("*.cuh")) + list(CSRC.glob("*.h")) + list(INCLUDE.glob("*.h"))


def up_to_date() -> bool:
    if not LIB.exists() or not CALLS.exists():
        return False
    t = min(LIB.stat().st_mtime, CALLS.stat().st_mtime)
    return all(p.stat().st_mtime <= t for p in _inputs())


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = False) -> Path:
    if not force and not ptxas_verbose and up_to_date():
        return LIB
    OUT.mkdir(exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", str(INCLUDE), "-I", str(CSRC)]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src: str):
        obj = OUT / (Path(src).stem + ".o")
        cmd = [nvcc, "-c", str(CSRC / src), "-o", str(obj)] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    failed = [(s, r) for s, _, r in results if r.returncode != 0]
    for s, _, r in results:
        if (ptxas_verbose or r.returncode != 0) and not quiet:
            sys.stderr.write(f"--- {s}\n{r.stdout}{r.stderr}")
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(s for s, _ in failed))
    tmp = OUT / "libdsv.so.tmp"
    cmd = [nvcc, "-shared", "-o", str(tmp)] + [str(o) for _, o, _ in results] + ARCH
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    tmp = CALLS.with_name(CALLS.name + ".tmp")
    cmd = [shutil.which("gcc") or "cc", "-shared", "-fPIC", "-O2", "-I", str(INCLUDE), "-I",
           sysconfig.get_paths()["include"], str(CSRC / "pycalls.c"), "-o", str(tmp), "-L", str(OUT), "-ldsv",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("building dsv_calls failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, CALLS)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv)
    print(LIB)
