"""Build of libpaged_decode.so: nvcc, one translation unit per head size,
compiled in parallel for sm_103a only, linked in-tree next to this file; and of
the Python module that marshals the step calls' arguments (bind.cpp)."""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpaged_decode.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")


def bind_path(python: str = sys.implementation.cache_tag, torch_version: str = torch.__version__) -> str:
    """The module of the step calls for a Python and a torch: it reads tensors by
    that torch's headers, so another's is another file."""
    return os.path.join(HERE, f"_bind.{python}-torch{torch_version}.so")


BIND = bind_path()
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fvisibility=hidden"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(os.path.dirname(HERE), "include", "*.h")))


def _bind_deps():
    return glob.glob(os.path.join(os.path.dirname(HERE), "include", "*.h")) + [BIND_SRC]


def _cxx():
    return shutil.which("g++") or shutil.which("c++")


def bind_missing() -> str:
    """What the module needs to be compiled and is not here ('' : nothing).  The
    library is built without it; the step calls then say so."""
    if not _cxx():
        return "a C++ compiler (g++ or c++)"
    for path in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                 os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd",
                              "python_variable.h")):
        if not os.path.exists(path):
            return path
    return ""


def _newer(target, deps) -> bool:
    """Was the target built after its last dependency changed?"""
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def bind_up_to_date() -> bool:
    return _newer(BIND, _bind_deps())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every .cu under csrc/ and link libpaged_decode.so, and compile the
    step calls' module beside it (a machine without a C++ compiler or the headers
    of Python or torch does without)."""
    lib, bind = force or not up_to_date(), force or not bind_up_to_date()
    missing = bind_missing() if bind else ""
    if missing:
        bind = False
        warnings.warn(f"the step calls are not built: {missing} is missing")
    if not lib and not bind:
        return LIB
    nvcc = _nvcc()
    inc = ["-I" + os.path.join(os.path.dirname(HERE), "include")]
    with cf.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        bound = ex.submit(_build_bind, nvcc, inc) if bind else None
        if lib:
            _build_lib(nvcc, inc, ex, verbose, extra_flags)
        if bound:
            bound.result()
    return LIB


def _build_bind(nvcc, inc):
    root = os.path.dirname(torch.__file__)
    tmp = BIND + f".tmp{os.getpid()}"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    cmd = [_cxx(), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc,
           "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(cuda, "include"), BIND_SRC, "-o", tmp, "-L" + os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed for bind.cpp:\n{r.stderr}")
    os.replace(tmp, BIND)


def _build_lib(nvcc, inc, ex, verbose, extra_flags):
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *inc, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
        return r.stderr

    logs = list(ex.map(compile_one, zip(srcs, objs)))
    if verbose:
        for lg in logs:
            if lg.strip():
                print(lg)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
