"""Builds libmuse.so (the C-ABI library) in-tree for sm_100a, and _torch_cache.so
(the paged-cache calls on torch tensors, a CPython module over libmuse.so).

    python -m clustered_multipole_approximation_b200.build [--force] [--ptxas-v]

Each .cu under csrc/ is compiled in parallel into _build/, then linked into
clustered_multipole_approximation_b200/libmuse.so next to this file.  The module
needs g++ and the headers of Python and torch; without them libmuse.so is built
all the same, with a warning.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmuse.so")
TORCH_SRC = os.path.join(CSRC, "torch_cache.cpp")
TORCH_LIB = os.path.join(PKG, "_torch_cache.so")
TORCH_KEY = TORCH_LIB + ".key"  # travels with the module

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libmuse")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _cxx() -> str:
    cxx = shutil.which("g++")
    if cxx is None:
        raise RuntimeError("g++ not found: it is needed to build _torch_cache.so")
    return cxx


def _torch_key() -> str:
    """What a built module belongs to: this torch and this Python."""
    import sysconfig

    import torch
    return "torch %s, %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def _torch_built_for():
    """The key of the module that is there; None where nothing says so."""
    if not os.path.exists(TORCH_KEY):
        return None
    with open(TORCH_KEY) as f:
        return f.read()


def _torch_stale() -> bool:
    """Whether the module is older than its sources."""
    t = os.path.getmtime(TORCH_LIB)
    return any(os.path.getmtime(p) > t for p in (TORCH_SRC, os.path.join(INCLUDE, "muse.h"), __file__))


def build_torch(force: bool = False) -> str:
    """The CPython module; libmuse.so has to stand next to it."""
    key = _torch_key()
    if not force and os.path.exists(TORCH_LIB) and not _torch_stale() and _torch_built_for() == key:
        return TORCH_LIB
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = TORCH_LIB + ".tmp.%d" % os.getpid()
    cmd = [_cxx(), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           TORCH_SRC, "-o", tmp, "-L", PKG, "-l:libmuse.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed on {TORCH_SRC}:\n{p.stderr}")
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_KEY, "w") as f:
        f.write(key)
    return TORCH_LIB


def _build_torch_or_warn(force: bool = False) -> None:
    """Every call but the paged cache's does without the module: where it cannot
    be compiled, libmuse.so stays usable.  A module of other sources or of another
    torch goes; one that nothing is known against stays."""
    try:
        build_torch(force)
    except (RuntimeError, OSError, ImportError) as e:
        if os.path.exists(TORCH_LIB):
            try:
                other = _torch_stale() or _torch_built_for() not in (None, _torch_key())
            except ImportError:
                other = True
            if not other:
                return
            os.remove(TORCH_LIB)
        warnings.warn(f"_torch_cache.so was not built, the paged-cache calls will raise: {e}", RuntimeWarning,
                      stacklevel=3)


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and up_to_date():
        _build_torch_or_warn()
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{p.stderr}")
        if ptxas_verbose:
            sys.stderr.write(p.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp.%d" % os.getpid()
    p = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"], capture_output=True,
                       text=True)
    if p.returncode != 0:
        raise RuntimeError("link failed:\n" + p.stderr)
    os.replace(tmp, LIB)
    _build_torch_or_warn(force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_verbose="--ptxas-v" in sys.argv)
    print(LIB)
