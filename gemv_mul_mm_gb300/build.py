"""Builds libqmm.so in-tree with nvcc for sm_103a (no cmake).

Each .cu translation unit compiles in parallel into an object, then one
link step makes the shared library. csrc/pycall.c, the CPython bindings of the
serving operators, becomes an extension module named for this Python's ABI;
without Python's headers the library is built all the same. Used by
``__graft_entry__.build()`` and by the Python binding when the library is
missing or stale.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqmm.so")
PYCALL_SRC = os.path.join(CSRC, "pycall.c")
PYCALL = os.path.join(HERE, "_pycall" + sysconfig.get_config_var("EXT_SUFFIX"))
ROOT = os.path.dirname(HERE)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(ROOT, "include", "qmm.h")]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in sources() + headers())


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--compiler-options", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"),
           *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build_pycall(force: bool = False) -> Optional[str]:
    """The extension module, or None where Python's headers or a C compiler are
    missing (qmm then says so when one of its operators is called)."""
    deps = [PYCALL_SRC, os.path.join(ROOT, "include", "qmm.h")]
    if not force and os.path.exists(PYCALL) and all(os.path.getmtime(f) <= os.path.getmtime(PYCALL) for f in deps):
        return PYCALL
    cc = next((c for c in (os.environ.get("CC"), shutil.which("gcc"), shutil.which("cc")) if c), None)
    include = sysconfig.get_paths()["include"]
    missing = "a C compiler" if cc is None else "" if os.path.exists(os.path.join(include, "Python.h")) else "Python.h"
    if missing:
        sys.stderr.write(f"{missing} not found: built without the Python bindings of qrope, qkv_store, qkv_load and qattn_decode\n")
        return None
    tmp = PYCALL + ".tmp"
    cmd = [cc, "-O2", "-Wall", "-fPIC", "-shared", "-fvisibility=hidden", "-I", include,
           "-I", os.path.join(ROOT, "include"), PYCALL_SRC, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cc} failed for pycall.c:\n{r.stderr}")
    os.replace(tmp, PYCALL)
    return PYCALL


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    lib = build_lib(force, verbose_ptxas)
    build_pycall(force)
    return lib


def build_lib(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
