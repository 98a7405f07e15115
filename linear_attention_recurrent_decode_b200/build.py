"""Build ``libkda_decode.so`` and ``libkda_layer.so`` in-tree with nvcc for sm_100a.

    python -m linear_attention_recurrent_decode_b200.build [--force] [-v]

``libkda_decode.so`` is the C ABI declared in ``include/kda_decode.h`` and
``include/kda_prefill.h`` (the CUDA translation units under ``csrc/``: one per
decode key size, the decode and prefill entry points); ``libkda_layer.so`` the
one under ``include/layer/`` (``csrc/layer/``: the operators of a layer around
the decode step, loaded on their first use).  The units are compiled in
parallel for ``sm_100a`` only and linked into one shared object per library,
with the CUDA runtime linked statically so it loads on its own (no torch, no
JIT cache).
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkda_decode.so")
OBJDIR = os.path.join(ROOT, "_build")
SOURCES = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
    os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
LAYER_LIB = os.path.join(PKG, "libkda_layer.so")
LAYER_CSRC = os.path.join(CSRC, "layer")
LAYER_INCLUDE = os.path.join(INCLUDE, "layer")
LAYER_SOURCES = sorted(os.path.join(LAYER_CSRC, f) for f in os.listdir(LAYER_CSRC) if f.endswith(".cu"))
LAYER_DEPENDS = LAYER_SOURCES + [os.path.join(LAYER_CSRC, f) for f in os.listdir(LAYER_CSRC) if f.endswith((".cuh", ".h"))] + [
    os.path.join(LAYER_INCLUDE, f) for f in os.listdir(LAYER_INCLUDE) if f.endswith(".h")] + [
    os.path.join(INCLUDE, "kda_decode.h"), os.path.join(CSRC, "kda_host_util.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def stale(lib: str = LIB, depends=None) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in (DEPENDS if depends is None else depends))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile each library that is missing or older than its sources; the decode library's path."""
    todo = [(lib, sources) for lib, sources, depends in ((LIB, SOURCES, DEPENDS), (LAYER_LIB, LAYER_SOURCES, LAYER_DEPENDS))
            if force or stale(lib, depends)]
    if not todo:
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    tag = f".{os.getpid()}"
    objs = {src: os.path.join(OBJDIR, os.path.basename(src)[:-3] + tag + ".o") for _, sources in todo for src in sources}

    def compile_one(src):
        cmd = [_nvcc(), *NVCC_FLAGS, "-c", "-I", INCLUDE, "-I", CSRC, "-o", objs[src], src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)

    try:
        with ThreadPoolExecutor(max_workers=max(1, min(len(objs), os.cpu_count() or 1))) as ex:
            list(ex.map(compile_one, objs))
        for lib, sources in todo:
            tmp = lib + f".tmp{os.getpid()}"
            subprocess.check_call([_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                                   "-Xcompiler", "-fPIC", "-o", tmp, *(objs[src] for src in sources)])
            os.replace(tmp, lib)
    finally:
        for o in objs.values():
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
