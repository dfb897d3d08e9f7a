"""Builds ``liblora_delta.so`` (the C ABI + sm_103a kernels) in-tree with nvcc.

Each translation unit compiles in its own nvcc process (in parallel), then
they are linked into one shared library next to this file. Only sm_103a code
is generated (one ``-gencode``). Rebuilds only when a source is newer than the
library.
"""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
CSRC_MLP = os.path.join(HERE, "csrc_mlp")     # the MLP-block operators (include/lora_mlp.h)
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "liblora_delta.so")
BUILD_DIR = os.path.join(os.path.dirname(HERE), "_build")
SOURCES = ["api.cu", "down.cu", "up.cu", "fwd_fused.cu", "fwd_cluster.cu", "bwd_cluster.cu", "dxda.cu", "wgrad.cu", "dy.cu", "rows.cu", "combine.cu", "noalloc.cu",
           "dvf32.cu", "exact.cu"]
SOURCES_MLP = ["host.cu", "layer_norm.cu", "pack8.cu", "pack8_da.cu", "gated_ffn.cu"]
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", *GENCODE]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _deps() -> list[str]:
    return [os.path.join(d, f) for d in (CSRC, CSRC_MLP, INCLUDE) for f in os.listdir(d)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags: tuple = (), lib: str = LIB) -> str:
    if not force and up_to_date(lib):
        return lib
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [cc, *NVFLAGS, *extra_flags, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    sources = [os.path.join(CSRC, f) for f in SOURCES] + [os.path.join(CSRC_MLP, f) for f in SOURCES_MLP]
    with ThreadPoolExecutor(max_workers=len(sources)) as ex:
        objs = list(ex.map(compile_one, sources))
    tmp = lib + ".tmp"
    cmd = [cc, "-shared", *GENCODE, "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True))
