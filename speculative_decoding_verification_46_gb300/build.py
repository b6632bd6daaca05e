"""Compile libspecverify.so in-tree for sm_103a with nvcc.

    python -m speculative_decoding_verification_46_gb300.build [--force]

The output goes to ``speculative_decoding_verification_46_gb300/lib/`` (git
ignored).  The library is rebuilt when a source or header is newer than it.
The verify step's sources are in ``csrc/``, those of the operators on logits
rows in ``rows/``, on the key/value cache in ``cache/``; the translation units
are compiled side by side.
"""

from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
ROWS = os.path.join(PKG, "rows")
CACHE = os.path.join(PKG, "cache")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIBNAME = "libspecverify.so"
LIB_PATH = os.path.join(LIBDIR, LIBNAME)

SOURCES = [os.path.join(CSRC, "sv_api.cu"), os.path.join(CSRC, "sv_noalloc.cu"), os.path.join(ROWS, "sv_rows_api.cu"),
           os.path.join(CACHE, "sv_cache_api.cu"), os.path.join(CACHE, "sv_attend_bf16.cu"),
           os.path.join(CACHE, "sv_attend_f16.cu")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _inputs():
    files = [os.path.join(d, f) for d in (CSRC, ROWS, CACHE) for f in os.listdir(d) if f.endswith((".cu", ".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _run_all(commands, verbose):
    """Run the commands at the same time; raise with the output of the first that fails."""
    running = []
    for cmd in commands:
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    results = [(proc, proc.communicate()[0]) for proc in running]
    for proc, output in results:
        if proc.returncode != 0:
            raise RuntimeError(f"nvcc failed ({proc.returncode}):\n{output}")


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build (if stale) and return the path of libspecverify.so."""
    if not force and os.path.exists(LIB_PATH):
        lib_mtime = os.path.getmtime(LIB_PATH)
        if all(os.path.getmtime(f) <= lib_mtime for f in _inputs()):
            return LIB_PATH
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    common = [_nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", f"-I{INCLUDE}"]
    objects = [f"{tmp}.{i}.o" for i in range(len(SOURCES))]
    commands = [[*common, "-c", src, "-o", obj] for src, obj in zip(SOURCES, objects)]
    try:
        _run_all(commands, verbose)
        _run_all([[*common, "-shared", "-o", tmp, *objects]], verbose)
    finally:
        for obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
