"""Build libcosa.so (the C-ABI library of the CUDA path) and libcosa_kv.so (what stands around it: include/cosa_kv.h)
in-tree for sm_103a.

Compiles the translation units under csrc/ in parallel with nvcc and links them into
block_sparse_long_gb300/libcosa.so and libcosa_kv.so.  The CUDA runtime is linked statically and the driver
API is reached through the runtime's entry-point query, so the libraries load on a machine
without a GPU (their calls then fail with COSA_ERR_CUDA).

    python -m block_sparse_long_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libcosa.so")
SOURCES = ["api.cu", "osk.cu", "osk_p16.cu", "osk_p32.cu", "osk_p64.cu", "osk_p128.cu", "osk_union_d64.cu",
           "osk_union_d128.cu", "kap.cu"]
HEADERS = ["ptx.cuh", "internal.h", "osk_kernel.cuh", "osk_union_kernel.cuh"]
KV_LIB = os.path.join(HERE, "libcosa_kv.so")
KV_SOURCES = ["kv_api.cu", "kv_rope.cu", "kv_convert.cu", "kv_attention.cu", "kv_evict.cu"]
KV_HEADERS = ["ptx.cuh", "kv_internal.h", "kv_layout.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (need the CUDA 13 toolkit)")
    return cand


def _inputs(sources, headers, public):
    files = [os.path.join(CSRC, s) for s in sources + headers]
    files += [os.path.join(ROOT, "include", h) for h in public]
    files.append(os.path.abspath(__file__))
    return files


# library, its translation units, the headers they include
LIBRARIES = ((LIB, SOURCES, HEADERS, ["cosa.h"]), (KV_LIB, KV_SOURCES, KV_HEADERS, ["cosa.h", "cosa_kv.h"]))


def _stale(lib, sources, headers, public) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in _inputs(sources, headers, public))


def up_to_date() -> bool:
    return not any(_stale(*entry) for entry in LIBRARIES)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the libraries whose inputs changed; returns the path of libcosa.so."""
    todo = [entry for entry in LIBRARIES if force or _stale(*entry)]
    if not todo:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    sources = [src for _, srcs, _, _ in todo for src in srcs]
    with ThreadPoolExecutor(len(sources)) as ex:
        objs = dict(zip(sources, ex.map(compile_one, sources)))
    for lib, srcs, _, _ in todo:
        tmp = lib + ".tmp"
        cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *(objs[src] for src in srcs)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
