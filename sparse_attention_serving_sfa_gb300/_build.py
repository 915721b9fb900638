"""Builds libsfa_gb300.so from csrc/*.cu with nvcc for sm_103a, and the module
_tensors (csrc/tensors.cpp: argument marshalling for torch tensors) with g++
against the installed torch's headers (both in-tree).  The library needs nvcc
alone: where the module cannot be built, a warning says why and the calls that
need it raise."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build", "sfa_gb300")
LIB_PATH = os.path.join(PKG, "libsfa_gb300.so")
TENSORS_SRC = os.path.join(CSRC, "tensors.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def tensors_path() -> str:
    """The _tensors module of this Python and torch (their C++ interfaces change
    between versions, so another pair builds its own)."""
    import sysconfig

    import torch
    tag = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    return os.path.join(PKG, f"_tensors_torch_{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _older(path, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(f) > os.path.getmtime(path) for f in deps)


def stale() -> bool:
    return _older(LIB_PATH, _deps())


def tensors_stale() -> bool:
    return _older(tensors_path(), [TENSORS_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))


def build_tensors() -> str:
    """Compile the _tensors module."""
    import sysconfig

    import torch
    where = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.sep in _nvcc() else "/usr/local/cuda"
    include = [os.path.join(where, "include"), os.path.join(where, "include/torch/csrc/api/include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(where, "lib")
    out = tensors_path()
    tmp = out + f".{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE,
           *[x for i in include for x in ("-isystem", i)],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-o", tmp, TENSORS_SRC,
           "-L", lib, f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(out):
            os.remove(out)              # an older module may not fit the library
        raise RuntimeError(f"g++ failed on tensors.cpp:\n{r.stderr}")
    os.replace(tmp, out)
    return out


def _try_tensors(force: bool) -> None:
    try:
        if force or tensors_stale():
            build_tensors()
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the library is built, the module for calls on torch tensors is not: {e}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every kernel source (in parallel) and link the shared library;
    compile the _tensors module beside it, if it can be."""
    if not force and not stale():
        _try_tensors(False)
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        tensors = ex.submit(_try_tensors, force)
        results = list(ex.map(compile_one, _sources()))
        tensors.result()
    if verbose:
        for _, log in results:
            print(log)
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
