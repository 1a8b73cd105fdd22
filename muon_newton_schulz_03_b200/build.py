"""Build the CUDA library ``libmuon_ns.so`` in-tree for sm_100a, and ``_lists.so``.

Usage: ``python -m muon_newton_schulz_03_b200.build [--force] [--verbose]``.

Compiles every ``csrc/*.cu`` / ``csrc/*.cpp`` with nvcc
(``-gencode arch=compute_100a,code=sm_100a -lineinfo -O3``) into one shared
library next to this file. Rebuilds only when a source or header is newer
than the library. The CUDA runtime is linked statically, so the library
loads without a GPU (entry points that need a device report
MUON_ERR_NO_DEVICE); no driver library is needed at link time.

``_lists.so`` (csrc/python/lists.cpp) is the part of the Python binding that
reads lists of torch tensors; it is compiled by the host compiler against the
installed torch, and again when that changes.
"""

from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmuon_ns.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
BUILD_DIR = os.path.join(HERE, "_build")
LISTS_SRC = os.path.join(CSRC, "python", "lists.cpp")
LISTS_PATH = os.path.join(HERE, "_lists.so")

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; set NVCC or put CUDA's bin directory on PATH")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                              + glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    if not force and not needs_build():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    flags = ARCH_FLAGS + COMMON_FLAGS + list(extra_flags or [])
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc, "-x", "cu", *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        objs.append(obj)
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _torch_version() -> str:
    from importlib.metadata import version
    return f"{version('torch')} {sys.version_info[:2]}"


def _lists_stamp() -> str:
    return os.path.join(BUILD_DIR, "lists.torch")


def lists_need_build() -> bool:
    if not os.path.exists(LISTS_PATH) or not os.path.exists(_lists_stamp()):
        return True
    t = os.path.getmtime(LISTS_PATH)
    with open(_lists_stamp()) as f:
        if f.read() != _torch_version():
            return True
    return any(os.path.getmtime(p) > t for p in (LISTS_SRC, os.path.join(INCLUDE, "muon_ns.h"), os.path.abspath(__file__)))


def build_lists(force: bool = False, verbose: bool = False) -> str:
    if not force and not lists_need_build():
        return LISTS_PATH
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    os.makedirs(BUILD_DIR, exist_ok=True)
    lib = os.path.join(home, "lib")
    tmp = f"{LISTS_PATH}.{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
           "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, LISTS_SRC, "-o", tmp, "-L", lib,
           f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on lists.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LISTS_PATH)
    with open(_lists_stamp(), "w") as f:
        f.write(_torch_version())
    return LISTS_PATH


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print register / shared-memory use (-Xptxas -v)")
    args = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if args.ptxas_info else []
    path = build(force=args.force or args.ptxas_info, verbose=args.verbose or args.ptxas_info, extra_flags=extra)
    print(path)
    print(build_lists(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    sys.exit(main())
