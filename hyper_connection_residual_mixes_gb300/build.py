"""Build libhc.so in-tree for GB300 (sm_103a) with nvcc.

Each .cu file under csrc/ is compiled in its own nvcc process (in parallel)
and the objects are linked into hyper_connection_residual_mixes_gb300/libhc.so.
The CUDA runtime is linked statically, so the library loads on a machine
without a GPU (its entry points then fail with HC_ERR_CUDA).

csrc/py_tensors.cpp becomes the Python module _tensors.so, with g++ beside them.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
TENSORS_SOURCE = os.path.join(CSRC, "py_tensors.cpp")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIB = os.path.join(PKG, "libhc.so")
TENSORS = os.path.join(PKG, "_tensors.so")
BUILD_DIR = os.path.join(PKG, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libhc")


def _gxx() -> str:
    cand = shutil.which("g++")
    if not cand:
        raise RuntimeError("g++ not found: it is required to build _tensors")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                              glob.glob(os.path.join(CSRC, "*.h")) +
                              glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(TENSORS)):
        return False
    t = os.path.getmtime(LIB)
    if _tensors_torch() != _torch_version():
        return False
    return (all(os.path.getmtime(p) <= t for p in _deps()) and
            os.path.getmtime(TENSORS_SOURCE) <= os.path.getmtime(TENSORS))


# the torch that _tensors was built for
_STAMP = os.path.join(BUILD_DIR, "tensors.torch")


def _tensors_torch():
    try:
        with open(_STAMP) as f:
            return f.read()
    except OSError:
        return None


def _torch_version():
    import torch
    return torch.__version__


def _build_tensors():
    import torch
    at = os.path.dirname(torch.__file__)
    tmp = TENSORS + ".tmp%d" % os.getpid()
    # (the torch libraries are loaded before the module is: no paths to them are kept)
    cmd = [_gxx(), "-O2", "-std=c++17", "-shared", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           '-DHC_TORCH_VERSION="%s"' % torch.__version__,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(at, "include"),
           "-isystem", os.path.join(at, "include", "torch", "csrc", "api", "include"), TENSORS_SOURCE, "-o", tmp,
           "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s%s" % (TENSORS_SOURCE, r.stdout, r.stderr))
    os.replace(tmp, TENSORS)
    with open(_STAMP, "w") as f:
        f.write(torch.__version__)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        tensors = ex.submit(_build_tensors)
        objs = list(ex.map(compile_one, srcs))
        tensors.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    # no -lcuda: driver entry points are fetched at run time through the
    # runtime, so the library also loads where no driver is installed.
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
