"""Build libaggemm.so (the CUDA library) in-tree with nvcc for sm_103a, and the native
part of the torch front end (_front, with Python's suffix for such modules), against the
installed torch, with g++.

The translation units compile in parallel; the results land next to this file.  A
rebuild happens only when a source or header is newer than a result, and for _front when
torch, Python or the machine is another than it was built for.  The library needs neither
torch nor g++: without torch _front is left out, and where building it fails the library
is in place before the error is raised.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libaggemm.so")
FRONT = os.path.join(HERE, "_front" + sysconfig.get_config_var("EXT_SUFFIX"))
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


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(result, inputs) -> bool:
    if not os.path.exists(result):
        return False
    t = os.path.getmtime(result)
    return all(os.path.getmtime(f) <= t for f in inputs)


def library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + _headers())


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _front_tag() -> str:
    """What a built _front belongs to (Python and the machine are in its suffix)."""
    import torch
    return torch.__version__ + " " + os.path.basename(FRONT)


def _stamp() -> str:
    return os.path.join(BUILD_DIR, "front.tag")


def front_up_to_date() -> bool:
    if not _newer(FRONT, [FRONT_SRC] + _headers()) or not os.path.exists(_stamp()):
        return False
    with open(_stamp()) as f:
        return f.read() == _front_tag()


def up_to_date() -> bool:
    return library_up_to_date() and (not _has_torch() or front_up_to_date())


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
    import torch
    os.makedirs(BUILD_DIR, exist_ok=True)
    obj = os.path.join(BUILD_DIR, "front.o")
    t = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-c", FRONT_SRC, "-o", obj, "-I" + INCLUDE,
          "-isystem", os.path.join(t, "include"),
          "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
          "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)], verbose)
    return obj


def _link_front(obj: str, verbose: bool = False) -> None:
    tmp = FRONT + ".%d.tmp" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN", *_torch_libs()], verbose)
    os.replace(tmp, FRONT)
    with open(_stamp(), "w") as f:
        f.write(_front_tag())


def build_library(verbose: bool = False) -> str:
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

    with ThreadPoolExecutor(max_workers=max(1, len(sources()))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [nvcc, "-shared", "-Xlinker", "-soname=libaggemm.so", *ARCH, "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, and _front where torch is installed.  Returns the library's path."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        front = None
        if _has_torch() and (force or not front_up_to_date()):
            front = ex.submit(_compile_front, verbose)
        if force or not library_up_to_date():
            build_library(verbose)
        if front:
            _link_front(front.result(), verbose)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
