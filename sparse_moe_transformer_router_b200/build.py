"""Build libl4moe.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m sparse_moe_transformer_router_b200.build [--force] [--verbose]

The CUDA runtime is linked statically and the driver API is reached through
cudaGetDriverEntryPoint, so the library has no link-time dependency on
libcuda (it loads on a machine without a GPU, e.g. for symbol checks).
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libl4moe.so")
OBJ = os.path.join(PKG, "build")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _includes(path: str, seen=None) -> set:
    """path and the package's own headers it includes, directly or not."""
    seen = set() if seen is None else seen
    if path in seen:
        return seen
    seen.add(path)
    with open(path) as f:
        for name in re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), re.M):
            for folder in (CSRC, INCLUDE):
                if os.path.exists(os.path.join(folder, name)):
                    _includes(os.path.join(folder, name), seen)
    return seen


def _made_by(nvcc: str, flags) -> str:
    """What an object is made by besides its sources: the compiler and the flags."""
    version = subprocess.run([nvcc, "--version"], capture_output=True, text=True, check=True).stdout
    return "\n".join([os.path.realpath(nvcc), version, *flags])


def _kept(src: str, obj: str, stamp: str, made_by: str) -> bool:
    """Whether obj is newer than all it includes and was made by the same compiler and flags."""
    if not (os.path.exists(obj) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        if f.read() != made_by:
            return False
    return all(os.path.getmtime(p) <= os.path.getmtime(obj) for p in _includes(src))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every source (side by side; one whose object is newer than all
    it includes, and made by the same compiler and flags, is kept) and link the
    library."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
             "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]
    nvcc = _nvcc()
    made_by = _made_by(nvcc, flags)
    if verbose:
        flags.insert(0, "-Xptxas=-v")
    jobs, objects = [], []
    for src in _sources():
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objects.append(obj)
        stamp = obj + ".made_by"
        if not force and _kept(src, obj, stamp, made_by):
            continue
        tmp = f"{obj}.tmp{os.getpid()}.o"
        cmd = [nvcc, *flags, "-c", src, "-o", tmp]
        jobs.append((cmd, tmp, obj, stamp,
                     subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = None
    for cmd, tmp, obj, stamp, p in jobs:
        out = p.communicate()[0]
        if verbose or p.returncode != 0:
            sys.stderr.write(out)
        if p.returncode != 0:
            failed = f"nvcc failed ({p.returncode}): {' '.join(cmd)}"
        else:
            if os.path.exists(stamp):  # (an object never stands beside another's stamp)
                os.remove(stamp)
            os.replace(tmp, obj)
            with open(stamp, "w") as f:
                f.write(made_by)
    if failed:
        raise RuntimeError(failed)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objects]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc failed ({r.returncode}): {' '.join(cmd)}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
