"""Build libpa_gb300.so in-tree with nvcc for sm_103a (GB300).

Each translation unit under csrc/ compiles in parallel; the objects link into
one shared library with the static CUDA runtime.  csrc/pa_pyfast.cpp, the
argument marshalling of q4.py and q8.py, becomes a Python extension beside it where the
interpreter's and torch's headers are installed (both work without it).  It reads
torch's tensors by their layout and calls the library by the headers' prototypes, so
its file is named by a digest of all that it was compiled from: one of other sources,
another torch or another interpreter is never loaded.  Usage:
    python -m paged_kv_gqa_pa_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import contextlib
import glob
import hashlib
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libpa_gb300.so")
PYFAST_SRC = os.path.join(CSRC, "pa_pyfast.cpp")
PYFAST_HEADERS = [os.path.join(ROOT, "include", h) for h in ("pa.h", "pa_q4.h", "pa_q8.h")]
PYFAST_FLAGS = ["-O2", "-std=c++17", "-shared", "-fPIC"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libpa_gb300.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _cuda_include():
    return os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")


def pyfast_path():
    """Where the marshalling extension of these sources, this torch and this interpreter lies,
    built or not; None without torch."""
    torch_dir = _torch_dir()
    version = os.path.join(torch_dir, "version.py") if torch_dir else ""  # (its git revision too)
    if not os.path.exists(version):
        return None
    h = hashlib.sha256(repr((sys.implementation.cache_tag, platform.machine(),
                             PYFAST_FLAGS)).encode())
    for path in [version, PYFAST_SRC, *PYFAST_HEADERS]:
        with open(path, "rb") as f:
            h.update(hashlib.sha256(f.read()).digest())
    return os.path.join(BUILD, f"_pa_fast-{h.hexdigest()[:16]}.so")


def _start_pyfast(force: bool, verbose: bool):
    """A running compilation of the marshalling extension and its output file; None if it is
    there, or without a C++ compiler or the interpreter's or torch's headers.  Extensions of
    other sources do not stay behind."""
    path = pyfast_path()
    for old in glob.glob(os.path.join(BUILD, "_pa_fast*.so")):
        if old != path:
            with contextlib.suppress(FileNotFoundError):  # (another build was first)
                os.remove(old)
    inc, torch_dir = sysconfig.get_paths()["include"], _torch_dir()
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if path is None or cxx is None or not os.path.exists(os.path.join(inc, "Python.h")):
        return None
    if not os.path.exists(os.path.join(torch_dir, "include", "torch", "csrc", "autograd",
                                       "python_variable.h")):
        return None
    if not force and os.path.exists(path):
        return None
    os.makedirs(BUILD, exist_ok=True)
    tmp = path + f".tmp{os.getpid()}"
    cmd = [cxx, *PYFAST_FLAGS, "-I", inc,
           "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-isystem", _cuda_include(), "-o", tmp, PYFAST_SRC,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd), tmp, path


def _finish_pyfast(job) -> None:
    if job is None:
        return
    proc, tmp, path = job
    if proc.wait() == 0:
        os.replace(tmp, path)
    else:
        print("the marshalling extension was not built; q4.py and q8.py go without it", file=sys.stderr)
        if os.path.exists(tmp):
            os.remove(tmp)


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    pyfast = _start_pyfast(force, verbose)
    try:
        return _build_lib(force, verbose, ptxas_verbose)
    finally:
        _finish_pyfast(pyfast)


def _build_lib(force: bool, verbose: bool, ptxas_verbose: bool) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or ptxas_verbose or p.returncode):
            sys.stderr.write(out)
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed on {failed}")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_verbose=a.ptxas_verbose))
