"""Build libq1gemv.so (the C-ABI library) from csrc/ with nvcc for sm_103a, and
_marshal.so (the operators' calls from Python, csrc/marshal.cpp) beside it.

    python -m decode_q1_gemv_gb300.build [--force] [--verbose]

Each translation unit compiles in parallel; the library lands in
decode_q1_gemv_gb300/_build/libq1gemv.so (git-ignored, rebuilt on every
machine: the output is architecture-specific).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libq1gemv.so")
MARSHAL = os.path.join(BUILD, "_marshal.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = [*ARCH, "-lineinfo", "-O3", "-std=c++17", "-fmad=false",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-ffp-contract=off",
              "-Xcompiler", "-fno-fast-math", "-I", INCLUDE]


MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + [MARSHAL_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "q1gemv.h")]


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return any(os.path.getmtime(p) > t for p in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    def compile_marshal():
        import torch

        root = os.path.dirname(torch.__file__)
        inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(cc)), "include"), INCLUDE]
        obj = os.path.join(BUILD, "marshal.o")
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", *(f"-I{p}" for p in inc), "-c", MARSHAL_SRC, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
        return obj, os.path.join(root, "lib")

    with cf.ThreadPoolExecutor(max_workers=min(9, (os.cpu_count() or 1) + 1)) as ex:
        marshal = ex.submit(compile_marshal)
        objs = list(ex.map(compile_one, sources()))
        marshal_obj, torch_lib = marshal.result()
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = MARSHAL + f".tmp{os.getpid()}"
    r = subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, marshal_obj, "-L" + BUILD, "-l:" + os.path.basename(LIB),
                        "-L" + torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN",
                        "-Wl,-rpath," + torch_lib], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
