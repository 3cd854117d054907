"""Build libaggemm.so (the CUDA library) in-tree with nvcc for sm_103a, and _front.so
(the native part of the torch front end, against the installed torch) with g++.

The translation units compile in parallel; the results land next to this file.  A
rebuild happens only when a source or header is newer than the results.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libaggemm.so")
FRONT = os.path.join(HERE, "_front.so")
FRONT_SRC = os.path.join(CSRC, "front.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libaggemm.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return (sources() + [FRONT_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(FRONT):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(FRONT))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _run(cmd, verbose=False):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _torch_libs():
    # (torch itself loads them first: importing it comes before the module)
    return ["-L" + os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
            "-lc10_cuda", "-lc10"]


def _compile_front(verbose: bool = False) -> str:
    import sysconfig
    import torch
    obj = os.path.join(BUILD_DIR, "front.o")
    t = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-c", FRONT_SRC, "-o", obj, "-I" + INCLUDE,
          "-isystem", os.path.join(t, "include"),
          "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
          "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)], verbose)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *CFLAGS, *ARCH, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=len(sources()) + 1) as ex:
        front = ex.submit(_compile_front, verbose)
        objs = list(ex.map(compile_one, sources()))
        front_obj = front.result()
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [nvcc, "-shared", "-Xlinker", "-soname=libaggemm.so", *ARCH, "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = FRONT + ".%d.tmp" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, front_obj, LIB, "-Wl,-rpath,$ORIGIN", *_torch_libs()], verbose)
    os.replace(tmp, FRONT)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
