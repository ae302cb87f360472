"""Builds librmsnorm_gb300.so in-tree from csrc/*.cu with nvcc for sm_103a, and
_binding.*.so, the native argument marshalling of api.py, from csrc/binding.cpp
with g++ against the installed torch (its version is part of the file's name).
The library needs nvcc alone; without torch the binding is left out.

Each translation unit compiles in its own nvcc process (in parallel), then
nvcc links them into one shared library with the CUDA runtime linked
statically, so the library needs only the driver at run time.  Rebuilds only
when a source or header is newer than the library.

    python -m rmsnorm_fwd_bwd_add_gb300.build [--force] [--verbose]
    python rmsnorm_fwd_bwd_add_gb300/build.py [--force] [--verbose]   # without torch
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
OBJ_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "librmsnorm_gb300.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "-I" + INCLUDE, "-I" + CSRC]


def binding_path() -> str:
    """The binding built for this torch and Python."""
    import torch
    return os.path.join(PKG_DIR, "_binding.%s.torch%s.so" % (
        sys.implementation.cache_tag, torch.__version__.replace("+", "_")))


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJ_DIR, os.path.basename(src).replace(".cu", ".o"))
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _binding_stale(path: str) -> bool:
    deps = [os.path.join(CSRC, "binding.cpp"), *glob.glob(os.path.join(INCLUDE, "*.h"))]
    return not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps)


def _binding_flags() -> list:
    import torch
    inc = [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(torch.__file__), "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]
    return ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(), *("-isystem" + i for i in inc)]


def _compile_binding(path: str) -> None:
    import torch
    tmp = path + ".tmp%d" % os.getpid()
    cmd = ["g++", *_binding_flags(), "-I" + INCLUDE, "-shared", os.path.join(CSRC, "binding.cpp"), "-o", tmp]
    cmd += ["-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on binding.cpp:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, path)


def _build_library(verbose: bool) -> None:
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB_PATH)


def _have_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library and, where torch is installed, the binding if
    needed; returns the library's path.  A binding that does not compile is raised
    once the library is linked."""
    binding = binding_path() if _have_torch() else None
    os.makedirs(OBJ_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside the library
        bound = ex.submit(_compile_binding, binding) if binding and (force or _binding_stale(binding)) else None
        if force or _stale(LIB_PATH):
            _build_library(verbose)
        if bound is not None:
            bound.result()
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/spill reports")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
