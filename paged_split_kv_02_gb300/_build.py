"""Build of libpaged_decode.so: nvcc, one translation unit per head size,
compiled in parallel for sm_103a only, linked in-tree next to this file; and of
the Python module that marshals the step calls' arguments (bind.cpp)."""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpaged_decode.so")
BIND = os.path.join(HERE, "_bind.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
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
            + glob.glob(os.path.join(os.path.dirname(HERE), "include", "*.h")) + [BIND_SRC])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BIND):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every .cu under csrc/ and link libpaged_decode.so."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    inc = ["-I" + os.path.join(os.path.dirname(HERE), "include")]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *inc, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
        return r.stderr

    def bind():
        import torch

        root = os.path.dirname(torch.__file__)
        libs = os.path.join(root, "lib")
        tmp = BIND + f".tmp{os.getpid()}"
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
        cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc,
               "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
               "-isystem", os.path.join(cuda, "include"), BIND_SRC, "-o", tmp, "-L" + libs,
               "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for bind.cpp:\n{r.stderr}")
        os.replace(tmp, BIND)

    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        bound = ex.submit(bind)
        logs = list(ex.map(compile_one, zip(srcs, objs)))
        bound.result()
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
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True))
