"""Build libmoe.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_marshal.so, the compiled argument marshalling of the dense operators' Python
entry points, with the host compiler.

Each .cu file under csrc/ is compiled in parallel to an object file under
_build/, then linked into grouped_gemm_top_gb300/libmoe.so.  Objects are
rebuilt only when a source or header is newer.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe")
    return cand


def _deps_mtime():
    files = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(f) for f in files), default=0.0)


def _compile(nvcc, src, obj, ptxas_verbose):
    cmd = [nvcc, *ARCH, *NVFLAGS, "-c", src, "-o", obj]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def build(verbose: bool = False, ptxas_verbose: bool = False, force: bool = False) -> str:
    """Compile every kernel source and link libmoe.so; returns its path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    dep_t = _deps_mtime()
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        stale = force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), dep_t)
        if stale:
            jobs.append((src, obj))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = {ex.submit(_compile, nvcc, s, o, ptxas_verbose): s for s, o in jobs}
            for fut in cf.as_completed(futs):
                log = fut.result()
                if verbose and log:
                    print(f"[{os.path.basename(futs[fut])}]\n{log}", file=sys.stderr)
    newest_obj = max(os.path.getmtime(o) for o in objs)
    if force or jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest_obj:
        tmp = LIB + ".tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _build_marshal(force)
    return LIB


def _build_marshal(force):
    """csrc/marshal.c against Python's headers and libmoe.so beside it.  Where
    there is no C compiler or Python has no headers, the library is built
    without it (and says so): the MoE layer does not need it."""
    src = os.path.join(CSRC, "marshal.c")
    there = os.path.exists(MARSHAL)
    fresh = there and os.path.getmtime(MARSHAL) >= max(os.path.getmtime(src), _deps_mtime())
    if fresh and not force:
        return
    cc, headers = shutil.which("gcc") or shutil.which("cc"), sysconfig.get_paths()["include"]
    if cc is None or not os.path.exists(os.path.join(headers, "Python.h")):
        if there and not fresh:
            os.remove(MARSHAL)      # older than the calls it makes
        print(f"_marshal.so not built: no {'C compiler' if cc is None else 'Python.h in ' + headers}; the dense "
              "operators (norm, linear, gated feed-forward, AdamW) need it", file=sys.stderr)
        return
    tmp = MARSHAL + ".tmp"
    cmd = [cc, "-O2", "-Wall", "-shared", "-fPIC", "-I", INCLUDE, "-I", headers, src, "-o", tmp, "-L", PKG,
           "-l:libmoe.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building _marshal.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(verbose=v, ptxas_verbose=v, force="--force" in sys.argv))
