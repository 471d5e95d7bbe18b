"""Build librom.so (the CUDA library of this package) in-tree for sm_100a.

    python -m mixture_experts_projections_b200.build [--verbose]

Compiles every csrc/*.cu with nvcc for sm_100a only, in parallel, and links
them (with the static CUDA runtime) into mixture_experts_projections_b200/
librom.so, and binding/fast_calls.cpp with g++ against the installed torch
into _fast_calls.so (where that cannot be built, rom.py checks its arguments in
Python). Objects go to mixture_experts_projections_b200/_build/.
Sources are rebuilt only when they, or a header under csrc/ or include/, changed.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librom.so")
FAST_SRC = os.path.join(PKG, "binding", "fast_calls.cpp")
FAST = os.path.join(PKG, "_fast_calls.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                 "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librom.so")


def _deps_mtime(src: str) -> float:
    """Newest mtime of the headers that `src` includes (transitively)."""
    seen, todo, newest = set(), [src], 0.0
    while todo:
        f = todo.pop()
        for inc in re.findall(r'#include\s+"([^"]+)"', open(f).read()):
            h = os.path.normpath(os.path.join(os.path.dirname(f), inc))
            if h not in seen and os.path.exists(h):
                seen.add(h)
                newest = max(newest, os.path.getmtime(h))
                todo.append(h)
    return newest


def _compile(src: str, verbose: bool, force: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if (not force and os.path.exists(obj)
            and os.path.getmtime(obj) >= max(os.path.getmtime(src), _deps_mtime(src))):
        return obj
    cmd = [nvcc()] + CFLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def _build_fast_calls(force: bool) -> None:
    """The binding's checked calls (a Python extension on torch's C++ API)."""
    if (not force and os.path.exists(FAST)
            and os.path.getmtime(FAST) >= max(os.path.getmtime(FAST_SRC), _deps_mtime(FAST_SRC))):
        return
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = include_paths() + [cuda_inc, sysconfig.get_paths()["include"]]
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wno-unknown-pragmas",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", FAST_SRC, "-o", FAST]
           + [f"-isystem{p}" for p in inc]
           + [f"-L{p}" for p in library_paths()] + ["-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {FAST_SRC}:\n{res.stdout}\n{res.stderr}")


def _try_build_fast_calls(force: bool) -> None:
    """The same where it can be built; an extension of older sources does not stay."""
    try:
        _build_fast_calls(force)
    except (RuntimeError, OSError, ImportError) as e:
        if os.path.exists(FAST):
            os.remove(FAST)
        warnings.warn(f"no {os.path.basename(FAST)}: {e}", RuntimeWarning)


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile and link librom.so and, where g++ and torch's headers allow it, the
    binding's extension; returns librom.so's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        fast = ex.submit(_try_build_fast_calls, force)
        objs = list(ex.map(lambda s: _compile(s, verbose, force), srcs))
        fast.result()
    if (force or not os.path.exists(LIB)
            or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", LIB] + objs
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/smem usage")
    ap.add_argument("--force", action="store_true")
    a = ap.parse_args()
    print(build(verbose=a.verbose, force=a.force))
