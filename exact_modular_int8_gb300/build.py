"""Build libresgemm.so (the C-ABI library) in-tree with nvcc for sm_103a.

Every translation unit under csrc/ (.cu, and host-only .cpp) is compiled in parallel and linked into
``_build/libresgemm.so`` next to this file.  A unit is rebuilt when it, a
header it includes, or this script is newer than its object file.
csrc/python/f8_call.c, the binding's native call path, and f8_grad.cpp, which reads
torch's autograd nodes, become the extension modules ``_build/f8_call.so`` and ``f8_grad.so``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libresgemm.so")
CALL_SRC = os.path.join(CSRC, "python", "f8_call.c")
CALL_LIB = os.path.join(BUILD, "f8_call.so")
GRAD_SRC = os.path.join(CSRC, "python", "f8_grad.cpp")
GRAD_LIB = os.path.join(BUILD, "f8_grad.so")
CC = os.environ.get("CC", "gcc")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(ROOT, "include", "resgemm.h"), os.path.abspath(__file__)]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_module(src, lib, command, *options):
    """A Python extension module of csrc/python (no CUDA in it)."""
    if not _stale(lib, [src, os.path.join(ROOT, "include", "resgemm.h"), os.path.abspath(__file__)]):
        return
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [*command, "-fPIC", "-shared", "-Wall", "-I", sysconfig.get_paths()["include"], src, "-o", tmp, *options]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{command[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


def _build_call():
    _build_module(CALL_SRC, CALL_LIB, [CC, "-O2"])


def _build_grad():
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    lib = os.path.join(torch, "lib")
    _build_module(GRAD_SRC, GRAD_LIB, [CXX, "-O1", "-std=c++20"], "-isystem", os.path.join(torch, "include"), "-L", lib,
                  "-lc10", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}")


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link; return the library path."""
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    headers = _headers()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        if not ptxas_info and not _stale(obj, [src] + headers):
            return obj, ""
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(len(sources), os.cpu_count() or 1))) as ex:
        modules = [ex.submit(f) for f in (_build_call, _build_grad)]
        results = list(ex.map(compile_one, sources))
        for m in modules:
            m.result()
    objs = [o for o, _ in results]
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv))
