"""Build ``libmoe_gb300.so`` in-tree for sm_103a with nvcc.

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into a
shared library next to this file, and ``csrc/binding.cpp`` into the Python
module ``_moe_binding`` beside it.  Objects are rebuilt only when a source or
header is newer.  Usage: ``python -m mixture_experts_layer_07_gb300.build``.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "obj")
LIB = os.path.join(PKG, "libmoe_gb300.so")
# the interpreter's ABI is part of the name: each version has its own file
BINDING = os.path.join(PKG, "_moe_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
           "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH") or "/usr/local/cuda"
    cand = os.path.join(home, "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found (set CUDA_HOME)")
    return found


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    cc = nvcc()
    jobs = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if _stale(obj, [src] + headers):
            cmd = [cc, *ARCH, *NVFLAGS, *extra_flags, "-c", src, "-o", obj]
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, flush=True)

    # the Python module: host code, compiled along with the kernels.  Without Python's headers
    # the library is built all the same, for the entry points that do not go through the module.
    src = os.path.join(CSRC, "binding.cpp")
    bind = None
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        print(f"no Python.h: {BINDING} is not built", file=sys.stderr, flush=True)
    elif _stale(BINDING, [src] + headers):
        bind = [cc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-cudart", "none", "-I",
                INCLUDE, "-I", sysconfig.get_paths()["include"], src, "-o", BINDING + ".tmp"]
        jobs.append(bind)

    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(run, jobs))
    if bind:
        os.replace(BINDING + ".tmp", BINDING)
        jobs.remove(bind)
    if jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
