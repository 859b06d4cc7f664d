"""Builds the HLA-2 CUDA library (libhla2.so) in-tree for sm_103a.

Every translation unit is compiled by nvcc in parallel, then linked into
``chunked_scan_mixer_gb300/_build/libhla2.so``.  Nothing is installed.  ``--debug`` builds
the bounds-checking variant (HLA2_DEBUG: global-memory indices checked against the buffer
extents, a failed check recorded and the access skipped; see hla2_debug_status) into
``chunked_scan_mixer_gb300/_build_debug/libhla2.so``.  The normal build also makes the Python module of
the short calls' host side (csrc/host_calls.cpp), which the binding goes without where it cannot be
built.

    python -m chunked_scan_mixer_gb300.build [--force] [--ptxas-v] [--debug]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libhla2.so")
HOST = os.path.join(BUILD, "_hla2_host.so")
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(BUILD_DEBUG, "libhla2.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the HLA-2 CUDA library cannot be built")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def host_stale(target: str, deps: list[str], torch_version: str) -> bool:
    """Whether the host module is older than its sources, or was built against another torch (named in a file beside it)."""
    if _stale(target, deps):
        return True
    try:
        with open(target + ".torch") as f:
            return f.read() != torch_version
    except OSError:
        return True


def build_host(force: bool = False) -> bool:
    """Compiles csrc/host_calls.cpp against the torch that is installed; False where that fails."""
    import sysconfig

    import torch

    src = os.path.join(CSRC, "host_calls.cpp")
    if not force and not host_stale(HOST, [src] + _headers(), torch.__version__):
        return True
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    include = [os.path.join(at, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
               os.path.join(ROOT, "include")]
    tmp = HOST + f".{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *("-I" + i for i in include), src, "-o", tmp, "-L" + os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        r = subprocess.CompletedProcess(cmd, 1, "", str(e))
    if r.returncode != 0:
        sys.stderr.write(f"host_calls.cpp was not built; the binding does without it:\n{r.stderr[-2000:]}\n")
        if os.path.exists(HOST):
            os.remove(HOST)
        return False
    os.replace(tmp, HOST)
    with open(HOST + ".torch", "w") as f:
        f.write(torch.__version__)
    return True


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int | None = None, debug: bool = False) -> str:
    nvcc = _nvcc()
    build_dir, lib = (BUILD_DEBUG, LIB_DEBUG) if debug else (BUILD, LIB)
    flags = NVCC_FLAGS + (["-DHLA2_DEBUG"] if debug else [])
    objdir = os.path.join(build_dir, "obj")
    os.makedirs(objdir, exist_ok=True)
    hdrs = _headers()
    srcs = sources()
    objs = []
    todo = []
    for s in srcs:
        o = os.path.join(objdir, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            todo.append((s, o))

    def compile_one(so):
        s, o = so
        cmd = [nvcc] + flags + (["-Xptxas", "-v"] if ptxas_verbose else []) + ["-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(s)}:\n{r.stderr}")
        return r.stderr

    host = None
    if not debug:
        host = cf.ThreadPoolExecutor(max_workers=1)
        host.submit(build_host, force)
    if todo:
        with cf.ThreadPoolExecutor(max_workers=jobs or min(len(todo), os.cpu_count() or 4)) as ex:
            for log in ex.map(compile_one, todo):
                if ptxas_verbose and log:
                    sys.stderr.write(log)
    if force or todo or _stale(lib, objs):
        tmp = lib + f".{os.getpid()}.tmp"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, lib)
    if host is not None:
        host.shutdown(wait=True)
    return lib


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true")
    ap.add_argument("--debug", action="store_true", help="the bounds-checking build (HLA2_DEBUG)")
    args = ap.parse_args()
    print(build(force=args.force, ptxas_verbose=args.ptxas_v, debug=args.debug))


if __name__ == "__main__":
    main()
