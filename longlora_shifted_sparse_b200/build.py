"""Builds libs2attn.so in-tree with nvcc for sm_100a (B200).

Each ``csrc/*.cu`` compiles to an object under ``_build/`` (rebuilt when it or a header is
newer), then nvcc links the shared library with the CUDA runtime linked statically. The torch
layer's serving calls (``csrc/serve_calls.cpp``) compile to ``_serve_calls.so`` beside it, against
torch's headers; without torch there is no torch layer, and the library alone is built.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "_build", "s2attn")
LIB = os.path.join(PKG, "libs2attn.so")
CALLS = os.path.join(PKG, "_serve_calls.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(OBJ, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    newest_header = max([os.path.getmtime(h) for h in _headers()] + [0.0])
    nvcc = _nvcc()
    flags = NVCC_FLAGS + list(extra_flags)

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        if force or not os.path.exists(obj) or \
                os.path.getmtime(obj) < max(os.path.getmtime(src), newest_header):
            cmd = [nvcc] + flags + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd))
            subprocess.check_call(cmd)
        return obj

    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources))
    if force or not os.path.exists(LIB) or \
            os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        if verbose:
            print(" ".join(cmd))
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    build_calls(force, verbose)
    return LIB


def build_calls(force: bool = False, verbose: bool = False) -> str | None:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    src, header = os.path.join(CSRC, "serve_calls.cpp"), os.path.join(ROOT, "include", "s2attn.h")
    if not force and os.path.exists(CALLS) and \
            os.path.getmtime(CALLS) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return CALLS
    torch = spec.submodule_search_locations[0]
    include = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda", "include")]
    tmp = CALLS + ".tmp.%d" % os.getpid()
    # torch's libraries are in the process already when it is imported; libs2attn.so lies beside it
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", src, "-o", tmp] + \
        ["-I" + p for p in include] + \
        ["-L" + PKG, "-l:libs2attn.so", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(torch, "lib"),
         "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, CALLS)
    return CALLS


if __name__ == "__main__":
    print(build(verbose=True))
