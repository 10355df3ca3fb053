"""Builds libsgemm_gb300.so in-tree with nvcc for sm_103a.

Each translation unit under ``csrc/`` compiles in parallel; the objects are then
linked into one shared library next to this file (``_lib/``).  The build is
skipped when the library is newer than every source and header.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
OUT_DIR = os.path.join(PKG_DIR, "_lib")
OBJ_DIR = os.path.join(OUT_DIR, "obj")
LIB_NAME = "libsgemm_gb300.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
FAST_SRC = os.path.join(PKG_DIR, "binding", "fast_calls.cpp")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", f"-I{INCLUDE}", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    files = sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + \
        [os.path.abspath(__file__)]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _newer(path: str, files) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path)
                                        for f in files)


def fast_path() -> str:
    """The binding for this Python and this torch: it fits no other."""
    import sysconfig

    import torch
    return os.path.join(OUT_DIR, f"_fast_calls-torch{torch.__version__}-"
                                 f"{sysconfig.get_config_var('SOABI')}.so")


def build_binding(force: bool = False) -> str:
    """Compile the binding of the usual calls (host code only, against the installed torch)."""
    path = fast_path()
    inputs = [FAST_SRC, os.path.join(INCLUDE, "sgemm.h"), os.path.abspath(__file__)]
    if not force and _newer(path, inputs):
        return path
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    os.makedirs(OUT_DIR, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    include = [INCLUDE, sysconfig.get_paths()["include"], cuda, *cpp_extension.include_paths()]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{d}" for d in include[1:]), f"-I{INCLUDE}", FAST_SRC, "-o", tmp,
           f"-L{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {FAST_SRC}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, path)
    return path


def _try_binding(force: bool) -> None:
    """The library is whole without the binding, which needs torch, Python's headers and a C++
    compiler; the operators that use it say that it is missing when they are called."""
    try:
        build_binding(force)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the binding of the 4-bit and norm operators was not built: {e}")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJ_DIR, os.path.basename(src).replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH_FLAGS, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        sys.stderr.write(res.stdout + res.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of the shared library."""
    if not force and up_to_date():
        _try_binding(False)
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        ex.submit(_try_binding, force)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
