"""Build libpagedkv.so (sm_100a) in-tree with nvcc and g++.

``python -m paged_kv_cache_480_b200.build`` (or :func:`build`) compiles every
CUDA translation unit for ``-gencode arch=compute_100a,code=sm_100a`` in
parallel and links them, with the host block manager, into
``paged_kv_cache_480_b200/libpagedkv.so`` (CUDA runtime linked statically).
Objects go to ``paged_kv_cache_480_b200/_build/``; a unit is rebuilt when it
or any header is newer than its object.  ``_fastcall.*.so`` beside it is a small
CPython extension through which the binding makes the calls that are issued
once a layer and step; where Python's headers are missing it is left out, and
those calls say so.
"""
import glob
import importlib.machinery
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
FASTCALL = os.path.join(PKG, "_fastcall" + importlib.machinery.EXTENSION_SUFFIXES[0])

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra", "-I", INCLUDE]


def _nvcc():
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(src, obj, headers):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(f) > t for f in [src] + headers)


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(force=False, verbose=False, extra_nvcc=()):
    """Compile and link the library; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    headers = _headers()
    jobs = []
    objs = []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(src, obj, headers):
            jobs.append([_nvcc()] + ARCH + NVCC_FLAGS + list(extra_nvcc) + ["-c", src, "-o", obj])
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cpp"))):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(src, obj, headers):
            jobs.append(["g++"] + CXX_FLAGS + ["-c", src, "-o", obj])
    if jobs:
        with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
            for out in ex.map(_run, jobs):
                if verbose and out.strip():
                    print(out)
    if force or jobs or not os.path.exists(LIB) or any(
            os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        _run([_nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    src, python = os.path.join(CSRC, "py", "fastcall.cpp"), sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(python, "Python.h")):
        print(f"no Python.h in {python}: {os.path.basename(FASTCALL)} is not built", file=sys.stderr)
    elif force or _stale(src, FASTCALL, glob.glob(os.path.join(INCLUDE, "*.h"))):
        tmp = FASTCALL + f".tmp{os.getpid()}"
        _run(["g++"] + CXX_FLAGS + ["-I", python, "-shared", "-o", tmp, src])
        os.replace(tmp, FASTCALL)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
