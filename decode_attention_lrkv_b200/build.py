"""Builds liblrkv.so and liblrkv_serve.so in-tree with nvcc for sm_100a.

    python -m decode_attention_lrkv_b200.build [--force] [--ptxas-v]

Every csrc/*.cu (liblrkv.so, include/lrkv.h) and csrc/serve/*.cu
(liblrkv_serve.so, include/lrkv_serve.h) is compiled to an object on its own
(in parallel, into _build/), then each library's objects are linked with the
static CUDA runtime, so the libraries carry no run-time path dependencies.
_serve_calls.so, the Python binding's fast path, is compiled with g++ against
torch's headers and Python's, and again when either of them changes; where that
fails there is a warning, and the binding does without.
"""
import concurrent.futures
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblrkv.so")
SERVE_CSRC = os.path.join(CSRC, "serve")
SERVE_LIB = os.path.join(PKG, "liblrkv_serve.so")
CALLS_SRC = os.path.join(SERVE_CSRC, "serve_calls.cpp")
CALLS_LIB = os.path.join(PKG, "_serve_calls.so")
CALLS_STAMP = os.path.join(OBJ, "serve_calls.made_for")

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


def _calls_inputs():
    return [CALLS_SRC, os.path.join(INCLUDE, "lrkv.h"), os.path.join(INCLUDE, "lrkv_serve.h"), os.path.abspath(__file__)]


def _calls_made_for():
    """What _serve_calls.so is compiled against beside its sources."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:   # a source tree
        import torch as module
        torch = module.__version__
    return f"torch {torch}, Python {sys.version}"


def _calls_current():
    if not _newer(CALLS_LIB, _calls_inputs()) or not os.path.exists(CALLS_STAMP):
        return False
    with open(CALLS_STAMP) as f:
        return f.read() == _calls_made_for()


def up_to_date():
    return _newer(LIB, _inputs()) and _newer(SERVE_LIB, _serve_inputs()) and _calls_current()


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


def _build_calls():
    import torch
    for old in (CALLS_STAMP, CALLS_LIB):   # what cannot be built again may not fit any more
        if os.path.exists(old):
            os.remove(old)
    home = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = CALLS_LIB + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(home, "include"), "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", cuda, "-I", INCLUDE, CALLS_SRC, "-o", tmp,
           "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    os.replace(tmp, CALLS_LIB)
    with open(CALLS_STAMP, "w") as f:
        f.write(_calls_made_for())


def build(force=False, verbose=False, extra=()):
    """Compile the libraries that are not newer than all their sources; returns liblrkv.so's path."""
    todo = [(lib, srcs) for lib, srcs, inputs in
            ((LIB, sources(), _inputs()), (SERVE_LIB, serve_sources(), _serve_inputs()))
            if force or not _newer(lib, inputs)]
    os.makedirs(OBJ, exist_ok=True)
    srcs = [s for _, part in todo for s in part]
    workers = max(1, min(len(srcs) + 1, os.cpu_count() or 1))
    with concurrent.futures.ThreadPoolExecutor(workers) as ex:
        calls = ex.submit(_build_calls) if force or not _calls_current() else None
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
    if calls is not None and (error := calls.exception()):
        warnings.warn(f"_serve_calls.so was not built, the binding marshals its calls in Python: {error}", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    ptx_v = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force or bool(ptx_v), verbose=True, extra=ptx_v))
