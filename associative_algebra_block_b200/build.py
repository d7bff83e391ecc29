"""Builds libaal.so in-tree with nvcc for sm_100a, and the binding's small
argument marshaller (_fastcall, a CPython extension) with the C compiler.

Usage: ``python -m associative_algebra_block_b200.build`` (or
``__graft_entry__.build()``).  The library is one translation unit
(``csrc/aal_lib.cu``) linked against the static CUDA runtime, so it loads on
a machine without a GPU driver; CUDA driver entry points it needs are fetched
at run time through the runtime.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libaal.so")
# named for the interpreter whose headers it is built with
FASTCALL = os.path.join(PKG, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(SRC, f) for f in os.listdir(SRC)
                  if f.endswith((".cu", ".h", ".cuh", ".c")))


def needs_build() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(FASTCALL):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(FASTCALL))
    deps = sources() + [os.path.join(INCLUDE, "aal.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [nvcc_path(), *ARCH_FLAGS, "-lineinfo", "-O3", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-cudart", "static", "-I", INCLUDE, "-I", SRC,
           "-o", tmp, os.path.join(SRC, "aal_lib.cu")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_fastcall()
    return LIB


def build_fastcall() -> str:
    """The binding's argument marshaller, a CPython extension in plain C."""
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        raise RuntimeError("no C compiler found")
    tmp = FASTCALL + ".tmp"
    subprocess.run([cc, "-O2", "-std=c11", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall", "-I",
                    sysconfig.get_paths()["include"], "-I", INCLUDE, "-o", tmp, os.path.join(SRC, "fastcall.c")],
                   check=True)
    os.replace(tmp, FASTCALL)
    untagged = os.path.join(PKG, "_fastcall.so")  # an older build's: any interpreter would import it
    if os.path.exists(untagged):
        os.remove(untagged)
    return FASTCALL


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
