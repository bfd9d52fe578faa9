"""Builds libmoe_gb300.so in-tree from csrc/*.cu with nvcc for sm_103a.

Each translation unit compiles in parallel (a few seconds each), then nvcc
links the shared library. Host code is compiled with hidden visibility so only
the MOE_API entry points of include/moe.h are exported. csrc/binding.c becomes
the CPython module _binding beside the library that it is linked to; where it
does not compile (no Python.h), the library alone is built, with a warning, and
the Python functions around the layer raise ImportError.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return exe


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "moe.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date(target: str = LIB) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if force or not up_to_date():
        _build_library(verbose, extra)
    if force or not up_to_date(BINDING):
        _build_binding()
    return LIB


def _build_library(verbose: bool, extra: list[str] | None) -> None:
    os.makedirs(BUILD, exist_ok=True)
    exe = nvcc()
    extra = extra or []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [exe, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr, flush=True)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [exe, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _build_binding() -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("gcc") or "cc", "-O2", "-Wall", "-shared", "-fPIC", "-fvisibility=hidden", "-I",
           sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.c"), "-o", tmp, "-L", PKG,
           "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.returncode != 0 and f"{r.stdout}\n{r.stderr}"
    except OSError as e:  # no compiler
        failed = str(e)
    if not failed:
        os.replace(tmp, BINDING)
        return
    if os.path.exists(BINDING):  # of an older source
        os.remove(BINDING)
    warnings.warn(f"_binding is not built: the functions around the layer and of its gradient will raise ImportError\n{failed}",
                  stacklevel=3)


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True, extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
