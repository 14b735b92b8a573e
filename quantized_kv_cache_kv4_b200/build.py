"""Build libkv4.so (the C-ABI library) in-tree for sm_100a with nvcc.

Usage: python -m quantized_kv_cache_kv4_b200.build [--verbose]
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkv4.so")
SOURCES = ["kv4_api.cu", "kv4_append.cu", "kv4_attention.cu", "kv4_baseline.cu", "kv4_noalloc.cu",
           "kv4_block8.cu", "kv4_block8_tile.cu", "kv4_evict.cu"]
HEADERS = ["kv4_device.cuh", "kv4_internal.h", "kv4_attn_common.cuh", "kv4_plan.cuh",
           "kv4_split.cuh", "kv4_block8.cuh"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def flags(verbose: bool = False):
    f = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-shared", "-Xcompiler", "-fPIC", "-cudart", "static",
         "-Xcompiler", "-fvisibility=default", "--expt-relaxed-constexpr"]
    if verbose:
        f += ["-Xptxas", "-v"]
    extra = os.environ.get("KV4_NVCC_FLAGS", "").split()
    return f + extra


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    deps.append(os.path.join(HERE, "..", "include", "kv4.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + flags(verbose) + [os.path.join(CSRC, s) for s in SOURCES] + ["-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
