"""Compile the CUDA library for sm_103a and its compiled binding, in-tree.

Produces ``online_softmax_attn_gb300/libattn_gb300.so`` from the ``csrc/*.cu``
translation units, compiled in parallel with nvcc (one ``-gencode``) and linked
with the static CUDA runtime, so the library needs no libcuda at load time
(driver entry points are resolved at run time). ``_calls.so``, the Python side of
the calls whose host time matters (``csrc/binding.cpp``), is compiled beside it by
g++ against the installed torch, and again when torch or Python change. The library
needs neither: where only the binding fails to compile, the library is linked before
the error is raised.

    python -m online_softmax_attn_gb300.build [--force] [--ptxas-verbose] [--debug]

``--debug`` builds ``libattn_gb300_debug.so`` instead, compiled with
``-DATTN_DEBUG``: the kernels check their store indices and shared-memory
offsets, record ATTN_DEVERR_DEBUG_INDEX in the device error word on a failed
check and skip that access (nothing traps).
"""
from __future__ import annotations

import argparse
import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libattn_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
CALLS_PATH = os.path.join(PKG, "_calls.so")
DEBUG_BUILD_DIR = os.path.join(PKG, "_build_debug")
DEBUG_LIB_PATH = os.path.join(PKG, "libattn_gb300_debug.so")

SOURCES = ["api.cu", "merge.cu", "decode.cu", "prefill_simt.cu", "prefill_tc.cu",
           "decode_static.cu", "host_prefill.cu", "cache_e4m3.cu", "decode_runs.cu",
           "decode_shared.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    env = os.environ.get("NVCC")
    if env:
        return env
    for cand in ("/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or install the CUDA toolkit)")


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, obj: str, ptxas_verbose: bool, debug: bool = False) -> str:
    cmd = [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if debug:
        cmd.append("-DATTN_DEBUG")
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
    return res.stderr if ptxas_verbose else ""


def _calls_key() -> str:
    """What a compiled binding depends on besides its sources."""
    import torch

    return "\n".join([torch.__version__, os.path.dirname(torch.__file__), sys.version,
                      str(torch._C._GLIBCXX_USE_CXX11_ABI), os.environ.get("CXX", "g++")])


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _compile_calls(src: str, out: str) -> str:
    """The compiled binding: a Python extension that uses torch's headers and
    the torch libraries of this interpreter, and no CUDA."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    tmp = out + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{d}" for d in inc], src, "-o", tmp, f"-L{os.path.join(root, 'lib')}", "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-ldl"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, out)
    return ""


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True,
          debug: bool = False) -> str:
    """Compile (if stale) and link the library (the -DATTN_DEBUG variant with
    ``debug``); returns its path."""
    build_dir = DEBUG_BUILD_DIR if debug else BUILD_DIR
    lib_path = DEBUG_LIB_PATH if debug else LIB_PATH
    os.makedirs(build_dir, exist_ok=True)
    headers = _headers()
    jobs = []
    objs = []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(build_dir, s.replace(".cu", ".o"))
        objs.append(obj)
        if force or ptxas_verbose or _stale(obj, [src, *headers]):
            jobs.append((src, obj))
    logs = []
    calls = os.path.join(CSRC, "binding.cpp")
    os.makedirs(BUILD_DIR, exist_ok=True)
    calls_key = os.path.join(BUILD_DIR, "calls.key")  # one binding for both variants
    calls_stale = (force or _stale(CALLS_PATH, [calls, os.path.join(INCLUDE, "attn.h")])
                   or _read(calls_key) != _calls_key())
    calls_job = None
    if jobs or calls_stale:
        workers = min(len(jobs) + 1, max(1, os.cpu_count() or 1))
        with concurrent.futures.ThreadPoolExecutor(workers) as ex:
            futs = [ex.submit(_compile, s, o, ptxas_verbose, debug) for s, o in jobs]
            if calls_stale:
                calls_job = ex.submit(_compile_calls, calls, CALLS_PATH)
            for f in futs:
                logs.append(f.result())
    if force or jobs or _stale(lib_path, objs):
        tmp = lib_path + ".tmp"
        cmd = [nvcc_path(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, lib_path)
    if calls_job is not None:
        calls_job.result()
        with open(calls_key, "w") as f:
            f.write(_calls_key())
    if ptxas_verbose or not quiet:
        for log in logs:
            if log:
                sys.stderr.write(log)
    return lib_path


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    ap.add_argument("--debug", action="store_true", help="build the -DATTN_DEBUG variant")
    a = ap.parse_args(argv)
    print(build(force=a.force, ptxas_verbose=a.ptxas_verbose, quiet=False, debug=a.debug))


if __name__ == "__main__":
    main()
