"""Build libmla.so (the C-ABI library) in-tree with nvcc for sm_103a, and _host.so,
the extension module that the Python calls around the decode go through.

    python -m mla_latent_kv_14_gb300.build        # or build() from Python

Translation units compile in parallel; the shared object lands next to this
file (``libmla.so``, git-ignored). CUDA runtime is linked statically, the
driver entry point for tensor maps is looked up at run time, so the library
loads on a machine without a GPU (argument checks work there; launches fail).
"""
from __future__ import annotations

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
LIB = os.path.join(HERE, "libmla.so")
HOST = os.path.join(HERE, "_host.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["mla_api.cu", "cache_api.cu"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                   "-I", os.path.join(ROOT, "include"), "-I", CSRC, "--expt-relaxed-constexpr",
                   "-DMLA_BUILD_SO"]


def _run(cmd, what: str, verbose: bool = False):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, flush=True)


def _compile_host(verbose: bool = False) -> str:
    """host_binding.cpp against the installed PyTorch's headers."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    obj = os.path.join(BUILD, "host_binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", os.path.join(CSRC, "host_binding.cpp"), "-o", obj,
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(base, "include"),
          "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(cuda, "include")], "g++", verbose)
    return obj


def _link_host(obj: str, verbose: bool = False):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = HOST + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python", "-ltorch_cpu",
          "-ltorch_cuda", "-lc10", "-lc10_cuda"], "link of _host.so", verbose)
    os.replace(tmp, HOST)


def build(verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = _flags() + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        _run(cmd, f"nvcc for {src}", verbose)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        host = ex.submit(_compile_host, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        tmp = LIB + ".tmp"
        _run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-Xlinker", "-soname=libmla.so", "-cudart", "static", "-lpthread", "-ldl", "-lrt"],
             "link", verbose)
        os.replace(tmp, LIB)
        # after the library, which needs neither g++ nor the headers of Python and PyTorch
        _link_host(host.result(), verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
