"""Build libsemmoe.so (every CUDA source, sm_103a) in-tree.

    python -m token_expert_routing_gb300.build [-v]

Each .cu file is compiled by its own nvcc process (in parallel) into
``_build/``; the objects are linked into ``libsemmoe.so`` next to this file, and the
Python entry points (binding.cpp) into ``_fast`` beside it.
Objects are rebuilt when their source or a header is newer.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsemmoe.so")
FAST = os.path.join(PKG, "_fast" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))  # the Python entry points
BINDING_OBJ = os.path.join(BUILD, "binding.o")
CXX = os.environ.get("CXX", "g++")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-Werror", "cross-execution-space-call",
              "-I" + INCLUDE, "-I" + CSRC] + ARCH


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cuda, "bin", "nvcc")
    return p if os.path.exists(p) else "nvcc"


def _stale(obj: str, deps: list[str]) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    nvcc = _nvcc()
    import torch
    torch_dir = os.path.dirname(torch.__file__)
    binding = None  # the Python entry points, compiled beside the CUDA sources
    src = os.path.join(CSRC, "binding.cpp")
    if _stale(BINDING_OBJ, [src, os.path.join(INCLUDE, "semmoe.h")]):
        inc = os.path.join(torch_dir, "include")
        cmd = [CXX, "-c", src, "-o", BINDING_OBJ, "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE, "-I" + inc,
               "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), "-I" + sysconfig.get_paths()["include"],
               "-I" + os.path.join(os.path.dirname(os.path.dirname(nvcc)) or "/usr/local/cuda", "include"),
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
        if verbose:
            print(" ".join(cmd), flush=True)
        binding = subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True)
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if _stale(obj, [src] + headers) or extra_flags:
            cmd = [nvcc, "-c", src, "-o", obj] + flags
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(sources), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, sources))
    if _stale(LIB, objs):
        cmd = [nvcc, "-shared", "-o", LIB] + objs + ARCH + ["-lcuda"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    if binding is not None:
        err = binding.communicate()[1]
        if binding.returncode != 0:
            raise RuntimeError(f"the binding did not build:\n{err}")
    if _stale(FAST, [BINDING_OBJ]):
        cmd = [CXX, "-shared", BINDING_OBJ, "-o", FAST, "-L" + PKG, "-l:libsemmoe.so", "-Wl,-rpath,$ORIGIN",
               "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"the binding did not link:\n{r.stdout}\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
