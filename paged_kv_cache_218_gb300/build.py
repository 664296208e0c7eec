"""Build libpa.so (the C-ABI library) from csrc/ with nvcc for sm_103a, and
the extension that marshals some of its calls' arguments (_pycall.so).

Each translation unit compiles in parallel to an object file under
``_build/`` at the repository root, then nvcc links the shared library into
this package directory.  Static cudart; the driver API is reached through
the runtime's entry-point query, so no -lcuda is needed.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpa.so")
PYCALL = os.path.join(PKG, "_pycall.so")  # CPython extension: argument marshalling
SOURCES = ["pa_api.cu", "pa_decode.cu", "pa_prefill.cu", "pa_hybrid.cu", "pa_cascade.cu",
           "pa_rope.cu", "pa_window_decode.cu", "pa_window_prefill.cu", "pa_block_manager.cpp"]
HEADERS = ["pa_internal.h", "pa_ptx.cuh", "pa_decode_body.cuh", "pa_prefill_body.cuh",
           "pa_window.h", "pa_window_ptx.cuh", os.path.join("..", "..", "include", "pa.h"),
           os.path.join("..", "..", "include", "pa_block_manager.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _torch() -> str:
    """torch's folder, found without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed: _pycall needs its headers")
    return spec.submodule_search_locations[0]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, h) for h in HEADERS]
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    relink = force or bool(jobs)
    # the extension's one source, beside them: torch's headers take it a while
    torch = _torch()
    cxx = os.environ.get("CXX", "g++")
    py_src = os.path.join(CSRC, "pa_pycall.cpp")
    py_obj = os.path.join(BUILD, "pa_pycall.o")
    cuda = os.path.dirname(os.path.dirname(nvcc)) if os.path.sep in nvcc else "/usr/local/cuda"
    if force or _stale(py_obj, [py_src, os.path.join(CSRC, "..", "..", "include", "pa.h"),
                                os.path.join(torch, "version.py")]):
        jobs.append([cxx, "-O2", "-std=c++17", "-fPIC", "-Wall",
                     "-I" + sysconfig.get_paths()["include"],
                     "-isystem", os.path.join(torch, "include"),
                     "-isystem", os.path.join(cuda, "include"), "-c", py_src, "-o", py_obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with concurrent.futures.ThreadPoolExecutor(max(1, len(jobs))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("compiler failed: " + " ".join(cmd))
    if relink or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    if force or _stale(PYCALL, [py_obj]):
        tmp = PYCALL + f".tmp{os.getpid()}"
        lib = os.path.join(torch, "lib")
        subprocess.run([cxx, "-shared", py_obj, "-o", tmp, "-L" + PKG, "-l:libpa.so", "-L" + lib,
                        "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
                        "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], check=True)
        os.replace(tmp, PYCALL)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
