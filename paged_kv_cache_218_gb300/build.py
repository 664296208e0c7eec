"""Build libpa.so (the C-ABI library) from csrc/ with nvcc for sm_103a, and,
where torch is installed, the extension that marshals some of its calls'
arguments for ``binding`` (_pycall, for this interpreter and this torch).

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
SUFFIX = sysconfig.get_config_var("EXT_SUFFIX")
PYCALL = os.path.join(PKG, "_pycall" + SUFFIX)  # CPython extension: argument marshalling
SOURCES = ["pa_api.cu", "pa_decode.cu", "pa_prefill.cu", "pa_hybrid.cu", "pa_cascade.cu",
           "pa_rope.cu", "pa_window_decode.cu", "pa_window_prefill.cu", "pa_beam_select.cu",
           "pa_beam_reorder.cu", "pa_shared_prefix.cu", "pa_block_manager.cpp"]
HEADERS = ["pa_internal.h", "pa_ptx.cuh", "pa_decode_body.cuh", "pa_prefill_body.cuh",
           "pa_window.h", "pa_window_ptx.cuh", "pa_beam.h", "pa_shared.h",
           os.path.join("..", "..", "include", "pa.h"),
           os.path.join("..", "..", "include", "pa_block_manager.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _torch():
    """torch's folder, found without importing it; None: not installed."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


class _Extension:
    """How _pycall is compiled and linked, and whether it has to be."""

    def __init__(self, torch: str, nvcc: str):
        cxx = os.environ.get("CXX", "g++")
        src, obj = os.path.join(CSRC, "pa_pycall.cpp"), os.path.join(BUILD, "pa_pycall" + SUFFIX + ".o")
        include, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
        cuda = os.path.dirname(os.path.dirname(nvcc)) if os.path.sep in nvcc else "/usr/local/cuda"
        self.compile = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall",
                        "-I" + sysconfig.get_paths()["include"], "-isystem", include,
                        "-isystem", os.path.join(cuda, "include"), "-c", src, "-o", obj]
        self.tmp = PYCALL + f".tmp{os.getpid()}"
        self.link = [cxx, "-shared", obj, "-o", self.tmp, "-L" + PKG, "-l:libpa.so", "-L" + lib,
                     "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
                     "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
        # what the present binary was built against, written behind it
        self.stamp = os.path.join(BUILD, "pa_pycall" + SUFFIX + ".txt")
        with open(os.path.join(torch, "version.py")) as f:
            self.key = torch + "\n" + sysconfig.get_paths()["include"] + "\n" + f.read()
        have = None
        if os.path.exists(self.stamp):
            with open(self.stamp) as f:
                have = f.read()
        self.stale = have != self.key or _stale(
            PYCALL, [src, os.path.join(CSRC, "..", "..", "include", "pa.h")])

    def finish(self) -> None:
        subprocess.run(self.link, check=True)
        os.replace(self.tmp, PYCALL)
        with open(self.stamp, "w") as f:
            f.write(self.key)


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
    ext = _Extension(torch, nvcc) if torch else None
    if ext is None:
        sys.stderr.write("torch is not installed: libpa.so is built, and _pycall, which the "
                         "Python binding needs, is not\n")
    elif force or ext.stale:
        jobs.append(ext.compile)
    else:
        ext = None

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = []
    with concurrent.futures.ThreadPoolExecutor(max(1, len(jobs))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                failed.append(cmd)
    if any(ext is None or cmd is not ext.compile for cmd in failed):
        raise RuntimeError("compiler failed: " + " ".join(failed[0]))
    if relink or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    if failed:  # the extension only: libpa.so stands
        raise RuntimeError("compiler failed: " + " ".join(failed[0]))
    if ext is not None:
        ext.finish()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
