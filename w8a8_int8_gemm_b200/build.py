"""Build the CUDA library libw8a8.so in-tree with nvcc (sm_100a only), and _calls.so, the part of the Python
binding that is native (g++, against the installed torch).

    python w8a8_int8_gemm_b200/build.py [--force]

Objects go to ``_build/`` at the repository root; the shared object is
written next to this file, where the Python binding loads it from.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libw8a8.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "binding.cpp")

SOURCES = ["api.cu", "quant.cu", "gemm_sm100.cu", "linear_noalloc.cu", "chain.cu", "qk_norm_rope.cu", "attention.cu",
           "attention_rows.cu", "attention_sm100.cu"]
HEADERS = ["internal.h", "sm100_ptx.cuh", "quant_row.cuh", "attention.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I" + INCLUDE,
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libw8a8.so")


def _newest_input() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "w8a8.h"), __file__]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)
    build_calls(force, verbose)
    return LIB


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """The native part of the binding; it finds libw8a8.so beside itself."""
    spec = importlib.util.find_spec("torch")  # (not imported: that takes longer than the rest)
    if spec is None:
        raise RuntimeError("torch not found: the Python binding is built against it")
    torch_dir = os.path.dirname(spec.origin)
    inputs = [CALLS_SOURCE, os.path.join(INCLUDE, "w8a8.h"), __file__,
              os.path.join(torch_dir, "version.py")]
    if not force and os.path.exists(CALLS) and os.path.getmtime(CALLS) >= max(map(os.path.getmtime, inputs)):
        return CALLS
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=1",
           "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           CALLS_SOURCE, "-o", tmp, "-L" + PKG, "-l:libw8a8.so", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, CALLS)
    return CALLS


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = [cc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC",
           "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=True))
    return 0


if __name__ == "__main__":
    sys.exit(main())
