"""Builds libhstu_b200.so in-tree with nvcc for sm_100a (B200).

    python -m hstu_jagged_pointwise_b200.build [--force] [--verbose]

and libhstu_cache_b200.so (the paged history cache and its scorer) beside it.

Each .cu under csrc/ (csrc/cache/ for the second library) compiles to an object in
csrc/_build/ (recompiled when it or any header is newer), then the objects link into
a shared library next to this file.  The two libraries share headers only, so each
exports exactly the functions of its own header in include/.  The CUDA runtime is linked statically; the TMA descriptor encoder
is fetched from the driver at run time, so no libcuda link is needed.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(CSRC, "_build")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libhstu_b200.so")
CACHE_CSRC = os.path.join(CSRC, "cache")
CACHE_LIB = os.path.join(HERE, "libhstu_cache_b200.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def _headers():
    return [h for d in (CSRC, CACHE_CSRC, INCLUDE) for e in ("*.cuh", "*.h") for h in glob.glob(os.path.join(d, e))]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _obj(src):
    prefix = "cache_" if os.path.dirname(src) == CACHE_CSRC else ""
    return os.path.join(OBJ, prefix + os.path.basename(src)[:-3] + ".o")


def _compile(src, verbose):
    obj = _obj(src)
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return obj, r.returncode, r.stdout + r.stderr, " ".join(cmd)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    parts = [(LIB, sorted(glob.glob(os.path.join(CSRC, "*.cu")))),
             (CACHE_LIB, sorted(glob.glob(os.path.join(CACHE_CSRC, "*.cu"))))]
    hdrs = _headers()
    todo = [s for _, srcs in parts for s in srcs if force or verbose or _stale(_obj(s), [s, *hdrs])]
    if todo:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(todo))) as ex:
            for obj, rc, out, cmd in ex.map(lambda s: _compile(s, verbose), todo):
                if out.strip() and (rc != 0 or verbose):
                    sys.stderr.write(out)
                if rc != 0:
                    raise RuntimeError(f"nvcc failed: {cmd}")
    for lib, srcs in parts:
        objs = [_obj(s) for s in srcs]
        if force or any(s in todo for s in srcs) or _stale(lib, objs):
            tmp = lib + f".tmp{os.getpid()}"
            cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
                raise RuntimeError(f"link failed: {' '.join(cmd)}")
            os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="pass -Xptxas -v (registers, spills)")
    a = ap.parse_args()
    print(build(a.force, a.verbose))
