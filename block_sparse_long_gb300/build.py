"""Build libcosa.so (the C-ABI library of the CUDA path), libcosa_kv.so (what stands around it: include/cosa_kv.h) and
libcosa_attn.so (dense attention beside it: include/cosa_attn.h) in-tree for sm_103a, and _attn_call, the Python module that
checks a call's tensors for the latter.

Compiles the translation units under csrc/ in parallel with nvcc and links them into
block_sparse_long_gb300/libcosa.so, libcosa_kv.so and libcosa_attn.so.  The CUDA runtime is linked statically and the driver
API is reached through the runtime's entry-point query, so the libraries load on a machine
without a GPU (their calls then fail with COSA_ERR_CUDA).

    python -m block_sparse_long_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
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
KV_HEADERS = ["ptx.cuh", "kv_internal.h", "kv_layout.cuh", "kv_angles.cuh"]
ATTN_LIB = os.path.join(HERE, "libcosa_attn.so")
ATTN_SOURCES = ["attn_api.cu", "attn_tma.cu", "attn_rope.cu", "attn_commit.cu", "attn_paged.cu", "attn_prefill.cu"]
ATTN_HEADERS = KV_HEADERS + ["attn_internal.h", "attn_tma.h", "attn_mma.cuh"]
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


# host code against PyTorch's headers: its suffix names the interpreter and the machine
CALL = os.path.join(HERE, "_attn_call" + sysconfig.get_config_var("EXT_SUFFIX"))
CALL_SOURCES = ["attn_binding.cpp"]
CALL_TORCH = os.path.join(BUILD, "attn_call.torch")      # the torch that it was compiled against

# library, its translation units, the headers they include
LIBRARIES = ((LIB, SOURCES, HEADERS, ["cosa.h"]), (KV_LIB, KV_SOURCES, KV_HEADERS, ["cosa.h", "cosa_kv.h"]),
             (ATTN_LIB, ATTN_SOURCES, ATTN_HEADERS, ["cosa.h", "cosa_kv.h", "cosa_attn.h"]))


def _stale(lib, sources, headers, public) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in _inputs(sources, headers, public))


def _torch_version() -> str:
    """What names the torch that is there, without importing it: its version file."""
    with open(os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "version.py")) as f:
        return f.read()


def _call_stale() -> bool:
    """The module reads tensors in place, by the headers of the torch that it was compiled against: another one needs another build."""
    if _stale(CALL, CALL_SOURCES, [], ["cosa.h", "cosa_attn.h"]) or not os.path.exists(CALL_TORCH):
        return True
    with open(CALL_TORCH) as f:
        return f.read() != _torch_version()


def up_to_date() -> bool:
    return not any(_stale(*entry) for entry in LIBRARIES) and not _call_stale()


def _build_call() -> None:
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(ROOT, "include"), os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = CALL + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", *(f"-I{d}" for d in include[:1]),
           *(f"-isystem{d}" for d in include[1:]), *(os.path.join(CSRC, f) for f in CALL_SOURCES), "-o", tmp,
           f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALL_SOURCES[0]}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)
    os.makedirs(BUILD, exist_ok=True)
    with open(CALL_TORCH, "w") as f:
        f.write(_torch_version())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the libraries whose inputs changed; returns the path of libcosa.so."""
    todo = [entry for entry in LIBRARIES if force or _stale(*entry)]
    call = force or _call_stale()
    if not todo:
        if call:
            _build_call()
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
    with ThreadPoolExecutor(len(sources) + 1) as ex:
        other = ex.submit(_build_call) if call else None
        objs = dict(zip(sources, ex.map(compile_one, sources)))
    for lib, srcs, _, _ in todo:
        tmp = lib + ".tmp"
        cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *(objs[src] for src in srcs)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if other is not None:
        other.result()      # (the libraries need nothing of it)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
