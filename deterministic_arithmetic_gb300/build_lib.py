"""Builds ``liblora_delta.so`` (the C ABI + sm_103a kernels) in-tree with nvcc, and ``_mlp.so``, the
compiled Python binding of include/lora_mlp.h, with the host compiler.

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
BINDING = os.path.join(HERE, "_mlp.so")
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
    outs = [lib] + ([BINDING] if lib == LIB else [])
    if not all(os.path.exists(o) for o in outs):
        return False
    t = min(os.path.getmtime(o) for o in outs)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _run(cmd: list[str], what: str, verbose: bool = False) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)


def _binding_object() -> str:
    """csrc_mlp/bind.cpp, compiled against torch's headers."""
    import sysconfig

    import torch

    t = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD_DIR, "bind.o")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
          "-isystem", sysconfig.get_paths()["include"], "-isystem", t,
          "-isystem", os.path.join(t, "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
          "-c", os.path.join(CSRC_MLP, "bind.cpp"), "-o", obj], "g++ on bind.cpp")
    return obj


def _link_binding(obj: str) -> None:
    """``_mlp.so`` from that object, against torch's libraries and, beside it, the library."""
    import torch

    _run([os.environ.get("CXX", "g++"), "-shared", "-o", BINDING + ".tmp", obj,
          "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
          "-ltorch", "-lc10_cuda", "-lc10", "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"],
         "link of _mlp.so")
    os.replace(BINDING + ".tmp", BINDING)


def build(force: bool = False, verbose: bool = False, extra_flags: tuple = (), lib: str = LIB) -> str:
    if not force and up_to_date(lib):
        return lib
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [cc, *NVFLAGS, *extra_flags, "-I", INCLUDE, "-c", src, "-o", obj]
        _run(cmd, f"nvcc on {src}", verbose)
        return obj

    sources = [os.path.join(CSRC, f) for f in SOURCES] + [os.path.join(CSRC_MLP, f) for f in SOURCES_MLP]
    bind = lib == LIB                  # a library built elsewhere (other flags) has no binding of its own
    with ThreadPoolExecutor(max_workers=len(sources) + 1) as ex:
        binding = ex.submit(_binding_object) if bind else None
        objs = list(ex.map(compile_one, sources))
        binding = binding.result() if bind else None
    tmp = lib + ".tmp"
    cmd = [cc, "-shared", *GENCODE, "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"]
    _run(cmd, "link")
    os.replace(tmp, lib)
    if bind:
        _link_binding(binding)
    return lib


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True))
