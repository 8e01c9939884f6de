"""Builds libra.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libra.so")
BIND = os.path.join(PKG, "_bind.so")       # Python binding of part of it (CPython and torch C++ API)
OBJDIR = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
          "-I", os.path.join(os.path.dirname(PKG), "include")]
# The prologue decides INT4 codes in fp32: no multiply-add contraction there.
PER_FILE = {"ra_prologue.cu": ["-fmad=false"]}
SOURCES = ["ra_host.cu", "ra_prologue.cu", "ra_attn_int4.cu", "ra_attn_int4_pair.cu", "ra_attn_bf16.cu",
           "ra_noalloc.cu", "ra_block.cu", "ra_norm_rope.cu", "ra_kv4.cu", "ra_attn_tiles.cu"]


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(os.path.dirname(PKG), "include", "ra.h"))
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _newer(o, [s] + headers):
            cmd = ["nvcc"] + ARCH + COMMON + PER_FILE.get(src, []) + ["-c", s, "-o", o]
            if verbose:
                cmd += ["-Xptxas", "-v"]
            subprocess.run(cmd, check=True)
    if force or _newer(LIB, objs):
        tmp = LIB + ".tmp"
        subprocess.run(["nvcc"] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs, check=True)
        os.replace(tmp, LIB)
    try:
        build_bind(force)
    except (OSError, subprocess.CalledProcessError) as e:
        # libra.so and what is bound by ctypes do not need it; the operators that do say so when they are called.
        warnings.warn(f"the compiled binding could not be built ({e}): the operators around the attention will not "
                      "be available", RuntimeWarning)
    return LIB


def build_bind(force: bool = False) -> str:
    """Compiles the binding against the installed torch and libra.so beside it; anew for another torch or Python."""
    import torch
    src = os.path.join(CSRC, "ra_bind.cpp")
    made_for = f"{torch.__version__} {os.path.dirname(torch.__file__)} {sys.version}"
    stamp = os.path.join(OBJDIR, "bind.txt")
    same = False
    if os.path.exists(stamp):
        with open(stamp) as f:
            same = f.read() == made_for
    if not force and same and not _newer(BIND, [src, os.path.join(os.path.dirname(PKG), "include", "ra.h")]):
        return BIND
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = BIND + ".tmp"
    try:
        subprocess.run(["g++", "-O2", "-std=c++20", "-shared", "-fPIC"] + [a for i in inc for a in ("-isystem", i)]
                       + [src, "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
                          "-lc10_cuda", "-lc10", "-L" + PKG, "-l:libra.so", "-Wl,-rpath,$ORIGIN"], check=True)
    except (OSError, subprocess.CalledProcessError):
        if os.path.exists(BIND):
            os.remove(BIND)   # rather none than one that does not fit
        raise
    os.replace(tmp, BIND)
    with open(stamp, "w") as f:
        f.write(made_for)
    return BIND


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
