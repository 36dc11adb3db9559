"""In-tree build of the CUDA library ``libdflash.so`` for sm_103a (GB300).

Each translation unit under ``csrc/`` compiles in parallel with nvcc; the
objects link into one shared library next to this file.  The CUDA runtime is
linked statically, so the library depends only on the driver.  ``csrc/calls.cpp``,
the CPython module that marshals the ragged-chunk calls, compiles beside it with
g++ against the headers of the installed torch.

    python -m context_kv_update_gb300.build            # build if stale
    python -m context_kv_update_gb300.build --force
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libdflash.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
CALLS_PATH = os.path.join(HERE, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Werror", "all-warnings"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libdflash.so")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "dflash.h"),
                                                                  os.path.abspath(__file__)]


def _older(path: str, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path)
                                           for p in deps)


def _calls_stale() -> bool:
    return _older(CALLS_PATH, [CALLS_SRC, os.path.join(INCLUDE, "dflash.h"),
                               os.path.abspath(__file__)])


def is_stale() -> bool:
    return _older(LIB_PATH, _deps()) or _calls_stale()


def _compile(src: str, extra=()) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if extra:
        sys.stderr.write(r.stderr)
    return obj


def _build_calls() -> None:
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = CALLS_PATH + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC",
           "-shared", "-fvisibility=hidden",
           f'-DDFLASH_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(at, "include"),
           "-isystem", os.path.join(cuda, "include"), CALLS_SRC, "-o", tmp,
           "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(_build_calls) if force or _calls_stale() else None
        if force or _older(LIB_PATH, _deps()):
            _build_lib(verbose_ptxas)
        # the library is there for the calls that need nothing else, even where the
        # module does not compile
        if calls:
            calls.result()
    return LIB_PATH


def _build_lib(verbose_ptxas: bool) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="--ptxas-v" in sys.argv)
    print(LIB_PATH)
