"""Build libsparse_attn.so in-tree with nvcc (sm_103a) and g++, and the native
calls of the torch classes beside it.

Translation units are compiled in parallel into ``_build/`` and linked into
``head_heterogeneous_block_gb300/_lib/libsparse_attn.so`` and, where there is a
torch with its headers and Python's, ``_lib/_calls.so``; the library is built
whatever becomes of the calls.  Rebuilds only what changed (by modification time
of sources and headers).
"""
from __future__ import annotations

import importlib.util
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
OBJ = os.path.join(ROOT, "_build", "obj")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libsparse_attn.so")
CALLS_SRC = os.path.join(PKG, "binding", "calls.cpp")
CALLS = os.path.join(LIB_DIR, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources():
    cu = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))
    cpp = sorted(f for f in os.listdir(CSRC) if f.endswith(".cpp"))
    return cu, cpp


def _newest_header() -> float:
    t = 0.0
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            if f.endswith((".h", ".cuh")):
                t = max(t, os.path.getmtime(os.path.join(d, f)))
    return t


def _torch():
    """The torch package's folder, found without importing it; None: there is
    none, or no headers to compile the native calls with."""
    spec = importlib.util.find_spec("torch")
    if not (spec and spec.submodule_search_locations):
        return None
    torch = spec.submodule_search_locations[0]
    for header in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                   os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h")):
        if not os.path.exists(header):
            sys.stderr.write(f"{header} is missing: PackedAttention, Rotary and PagePool are not "
                             "built\n")
            return None
    return torch


def _compile(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    return cmd, r


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    nvcc = _nvcc()
    cu, cpp = _sources()
    hdr = _newest_header()
    jobs, objs = [], []
    common = ["-O3", "-std=c++17", f"-I{INCLUDE}", f"-I{CSRC}"]
    for f in cu:
        src = os.path.join(CSRC, f)
        obj = os.path.join(OBJ, f + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr):
            jobs.append([nvcc, *ARCH, "-lineinfo", *common, "-Xcompiler", "-fPIC",
                         "-Xptxas", "-v" if verbose else "-O3", "-c", src, "-o", obj])
    for f in cpp:
        src = os.path.join(CSRC, f)
        obj = os.path.join(OBJ, f + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr):
            jobs.append(["g++", *common, "-fPIC", "-Wall", "-c", src, "-o", obj])
    torch = _torch()
    calls_obj = os.path.join(OBJ, "calls.o")
    newest = max(os.path.getmtime(CALLS_SRC), hdr)
    if torch is None:
        # (calls of another library are not left beside the new one)
        if os.path.exists(CALLS) and os.path.getmtime(CALLS) < newest:
            os.remove(CALLS)
    else:
        newest = max(newest, os.path.getmtime(os.path.join(torch, "version.py")))
        if force or not os.path.exists(calls_obj) or os.path.getmtime(calls_obj) < newest:
            dirs = [sysconfig.get_paths()["include"], os.path.join(torch, "include"),
                    os.path.join(torch, "include", "torch", "csrc", "api", "include")]
            # (first: it takes as long as the largest kernel)
            jobs.insert(0, ["g++", "-O2", "-std=c++17", f"-I{INCLUDE}",
                            *(f"-isystem{d}" for d in dirs), "-fPIC", "-Wall", "-c", CALLS_SRC,
                            "-o", calls_obj])
    failed = []
    if jobs:
        with ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
            results = list(ex.map(_compile, jobs))
        failed = [(c, r) for c, r in results if r.returncode != 0]
        for c, r in results:
            if verbose or r.returncode != 0:
                sys.stderr.write(" ".join(c) + "\n" + r.stdout + r.stderr)
        if any(c[-1] != calls_obj for c, _ in failed):
            raise RuntimeError("compilation failed: " + next(
                os.path.basename(c[-3]) for c, _ in failed if c[-1] != calls_obj))
    if jobs or not os.path.exists(LIB):
        link = [nvcc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(LIB + ".tmp", LIB)
    if failed:
        if os.path.exists(CALLS):
            os.remove(CALLS)
        raise RuntimeError(f"compilation failed: {os.path.basename(CALLS_SRC)}")
    if torch is not None and (jobs or not os.path.exists(CALLS)):
        lib = os.path.join(torch, "lib")
        link = ["g++", "-shared", "-o", CALLS + ".tmp", calls_obj, f"-L{LIB_DIR}",
                "-l:libsparse_attn.so", "-Wl,-rpath,$ORIGIN", f"-L{lib}", "-ltorch_python",
                "-ltorch_cpu", "-lc10"]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(CALLS + ".tmp", CALLS)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
