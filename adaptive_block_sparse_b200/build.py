"""Builds ``libnabla.so`` (the C-ABI library) in-tree with nvcc for sm_100a.

Usage: ``python -m adaptive_block_sparse_b200.build`` (or ``build()`` from Python).
Each ``csrc/*.cu`` is compiled in parallel to an object file under ``_build/``; the
objects are linked into ``adaptive_block_sparse_b200/libnabla.so`` with the CUDA runtime
linked statically, so the library depends only on the NVIDIA driver at run time.
``csrc/binding.cpp`` (argument marshalling from torch tensors, host code) is compiled against
the installed torch into the Python module ``_binding.so`` beside it.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libnabla.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _compile(src: str, verbose: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest_dep = max(os.path.getmtime(p) for p in [src] + _headers())
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep and not extra:
        return obj
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr, flush=True)
    return obj


def _run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _compile_binding(verbose: bool) -> str:
    obj = os.path.join(BUILD, "binding.cpp.o")
    deps = [BINDING_SRC, os.path.join(INCLUDE, "nabla.h"), os.path.join(_torch_dir(), "version.py")]
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(p) for p in deps):
        return obj
    import torch
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-isystem", sysconfig.get_paths()["include"], "-c", BINDING_SRC, "-o", obj], "binding.cpp", verbose)
    return obj


def _link_binding(obj: str, verbose: bool) -> None:
    if os.path.exists(BINDING) and os.path.getmtime(BINDING) >= os.path.getmtime(obj):
        return
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libnabla.so", "-L", lib, "-ltorch_python", "-ltorch",
          "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,$ORIGIN,-rpath,{lib}"], "linking the binding", verbose)
    os.replace(tmp, BINDING)


def _link(objs, verbose: bool, extra) -> None:
    if (os.path.exists(LIB) and not extra and
            os.path.getmtime(LIB) >= max(os.path.getmtime(o) for o in objs)):
        return
    tmp = LIB + ".tmp"
    _run([nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-lrt", "-ldl", "-lpthread"],
         "linking the library", verbose)
    os.replace(tmp, LIB)


def build(verbose: bool = False, extra=()) -> str:
    """Compile every CUDA source, link ``libnabla.so`` and build ``_binding.so``; returns the
    library's path.  The library is there even if the binding cannot be built (a C program needs
    neither it nor torch's headers); that is raised afterwards."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose, list(extra)), srcs))
        _link(objs, verbose, extra)
        binding_obj = binding.result()
    _link_binding(binding_obj, verbose)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, extra=[a for a in sys.argv[1:] if a != "-v"])
    print(LIB)
