"""Builds liblrkv.so and liblrkv_serve.so in-tree with nvcc for sm_100a.

    python -m decode_attention_lrkv_b200.build [--force] [--ptxas-v]

Every csrc/*.cu (liblrkv.so, include/lrkv.h) and csrc/serve/*.cu
(liblrkv_serve.so, include/lrkv_serve.h) is compiled to an object on its own
(in parallel, into _build/), then each library's objects are linked with the
static CUDA runtime, so the libraries carry no run-time path dependencies.
"""
import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblrkv.so")
SERVE_CSRC = os.path.join(CSRC, "serve")
SERVE_LIB = os.path.join(PKG, "liblrkv_serve.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden"]


def nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build liblrkv.so")
    return exe


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def serve_sources():
    return sorted(glob.glob(os.path.join(SERVE_CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + \
        [os.path.join(INCLUDE, "lrkv.h"), os.path.abspath(__file__)]


def _inputs():
    return sources() + _headers()


def _serve_inputs():
    return serve_sources() + sorted(glob.glob(os.path.join(SERVE_CSRC, "*.cuh"))) + _headers() + \
        [os.path.join(INCLUDE, "lrkv_serve.h")]


def _newer(lib, inputs):
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in inputs)


def up_to_date():
    return _newer(LIB, _inputs()) and _newer(SERVE_LIB, _serve_inputs())


def _compile(src, extra):
    obj = os.path.join(OBJ, os.path.relpath(src, CSRC).replace(os.sep, "_")[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return obj, cmd, r


def _link(objs, lib):
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fvisibility=hidden", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, lib)


def build(force=False, verbose=False, extra=()):
    """Compile the libraries that are not newer than all their sources; returns liblrkv.so's path."""
    todo = [(lib, srcs) for lib, srcs, inputs in
            ((LIB, sources(), _inputs()), (SERVE_LIB, serve_sources(), _serve_inputs()))
            if force or not _newer(lib, inputs)]
    os.makedirs(OBJ, exist_ok=True)
    srcs = [s for _, part in todo for s in part]
    workers = max(1, min(len(srcs), os.cpu_count() or 1))
    with concurrent.futures.ThreadPoolExecutor(workers) as ex:
        results = dict(zip(srcs, ex.map(lambda s: _compile(s, list(extra)), srcs)))
    for obj, cmd, r in results.values():
        if verbose:
            print(" ".join(cmd))
            if r.stdout or r.stderr:
                print(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    for lib, part in todo:
        _link([results[s][0] for s in part], lib)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    ptx_v = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force or bool(ptx_v), verbose=True, extra=ptx_v))
