"""Builds libdsa_b200.so and its binding _gqa.so in-tree, with nvcc for sm_100a.

Every .cu file under csrc/ is compiled separately (in parallel) and linked
into one shared library that exports only the C ABI of include/dsa_b200.h.
The CUDA runtime is linked statically and its symbols are hidden.  _gqa.so is
the compiled part of the Python binding (csrc/gqa_binding.cpp, against torch's
C++ interface); it calls the library beside it.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libdsa_b200.so")
BINDING_SRC = os.path.join(CSRC, "gqa_binding.cpp")
BINDING_PATH = os.path.join(PKG, "_gqa.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                     "-Xcompiler", "-fPIC,-fvisibility=hidden,-O3", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(INCLUDE, "dsa_b200.h"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    return _newer(LIB_PATH, _deps()) and _binding_up_to_date()


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def _binding_up_to_date() -> bool:
    return _newer(BINDING_PATH, [BINDING_SRC, os.path.join(INCLUDE, "dsa_b200.h"), os.path.abspath(__file__)])


def build_binding(force: bool = False) -> str:
    """Compiles _gqa.so (g++, torch's headers); libdsa_b200.so must be there."""
    if not force and _binding_up_to_date():
        return BINDING_PATH
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        cmd += ["-isystem" if d != INCLUDE else "-I", d]
    lib = os.path.join(root, "lib")
    cmd += [BINDING_SRC, "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-L", PKG, "-l:libdsa_b200.so", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(BINDING_SRC)}:\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    if not force and _newer(LIB_PATH, _deps()):
        build_binding()
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [cc] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose or ptxas_info:
            print(r.stderr, end="")
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-Xlinker", "--exclude-libs,ALL"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    build_binding(force)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
