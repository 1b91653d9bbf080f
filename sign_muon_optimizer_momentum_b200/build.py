"""Builds libsignmuon.so in-tree with nvcc for sm_100a, and on top of it the
Python binding of layers.py (_layers_native.so, host code only).

Usage: ``python -m sign_muon_optimizer_momentum_b200.build`` (or through
``__graft_entry__.build()``).  Both are rebuilt only when a source or header is
newer than one of them.  The library needs nvcc alone: where PyTorch or
Python's headers are not installed it is built without the binding.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsignmuon.so")
BINDING = os.path.join(PKG, "_layers_native.so")
BINDING_SOURCE = os.path.join(CSRC, "layers_binding.cpp")
SOURCES = ["api.cu", "elementwise.cu", "ns_gemm.cu", "noalloc.cu", "embedding.cu", "layer_norm.cu", "distill.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libsignmuon.so")
    return nvcc


def _compile_binding(verbose: bool) -> str:
    """Object file of the PyTorch binding (g++; PyTorch's headers and flags)."""
    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(BUILD, "layers_binding.o")
    dirs = [INCLUDE, *cpp_extension.include_paths("cuda"), sysconfig.get_paths()["include"]]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++20", "-fPIC", "-DTORCH_API_INCLUDE_EXTENSION_H",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{d}" for d in dirs],
           "-c", BINDING_SOURCE, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on layers_binding.cpp")
    return obj


def _binding_can_be_built() -> bool:
    headers = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    return importlib.util.find_spec("torch") is not None and os.path.exists(headers)


def _link_binding(obj: str) -> None:
    import torch
    tmp = BINDING + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-lsignmuon", "-Wl,-rpath,$ORIGIN",
           f"-L{os.path.join(os.path.dirname(torch.__file__), 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("link of _layers_native.so failed")
    os.replace(tmp, BINDING)


def _newest_input() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    with_binding = _binding_can_be_built()
    made = (LIB, BINDING) if with_binding else (LIB,)
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= _newest_input() for f in made):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose or ptxas_info:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, verbose) if with_binding else None
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("link of libsignmuon.so failed")
    os.replace(tmp, LIB)
    if binding is None:
        sys.stderr.write("PyTorch or Python's headers are missing: built libsignmuon.so without the binding of layers.py\n")
    else:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv))
