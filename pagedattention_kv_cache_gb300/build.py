"""Build libpagedkv.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel to an object file under
``_build/``, then nvcc links them into ``pagedattention_kv_cache_gb300/libpagedkv.so``.
Usage: ``python -m pagedattention_kv_cache_gb300.build`` (or ``build()``).
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libpagedkv.so")
SOURCES = ["api.cu", "kv_store.cu", "decode.cu", "decode_mod.cu", "verify.cu", "fp8.cu", "blocks.cu", "prefill.cu",
           "prefill_tc.cu", "prefill_tc_masked.cu", "prefill_tc_capped.cu", "prefill_tc_biased.cu",
           "prefill_tc_capped_biased.cu", "prefill_tc_fp8.cu", "prefill_chunk.cu", "chunk_decode.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libpagedkv.so")


def _run(cmd: list[str]) -> None:
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"command failed ({proc.returncode}): {' '.join(cmd)}\n{proc.stdout}\n{proc.stderr}")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source and link the shared library; returns its path."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "pagedkv.h"))
    jobs = []
    objects = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objects.append(obj)
        if force or _stale(obj, [path] + headers):
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", path, "-o", obj])
    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs)) as pool:
            for fut in [pool.submit(_run, j) for j in jobs]:
                fut.result()
    if force or jobs or _stale(LIB_PATH, objects):
        tmp = LIB_PATH + ".tmp"
        _run([nvcc, *ARCH, "-shared", "-o", tmp, *objects])
        os.replace(tmp, LIB_PATH)
    if verbose:
        print(f"built {LIB_PATH}", file=sys.stderr)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
