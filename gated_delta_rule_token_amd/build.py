"""Build libgdr.so (the HIP kernels + C ABI) in-tree with hipcc for gfx950.

    python -m gated_delta_rule_token_amd.build

Each translation unit under ``csrc/`` is compiled to an object in
``_build/`` (in parallel), then linked into ``gated_delta_rule_token_amd/libgdr.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgdr.so")
ARCH = os.environ.get("GDR_OFFLOAD_ARCH", "gfx950")

SOURCES = ["gdr_api.cpp", "gdr_decode.hip", "gdr_recurrent.hip", "gdr_chunked.hip", "gdr_chunked_bf16.hip",
           "gdr_gate.hip", "gdr_stream.hip", "gdr_backward.hip", "gdr_backward_f32.hip", "gdr_backward_f16.hip",
           "gdr_backward_bf16.hip", "gdr_norm.hip", "gdr_rotary.hip", "gdr_packed.hip", "gdr_packed_f16.hip",
           "gdr_packed_bf16.hip", "gdr_packed_e4m3.hip"]

# Packed fp32 VALU forms are switched off for the device code; every kernel
# is ordinary fp32 arithmetic.
HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=" + ARCH,
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
    "-I" + INCLUDE, "-I" + CSRC,
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found; the HIP library cannot be built")
    return path


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc(), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj] + HIPCC_FLAGS
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed on %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr[-6000:]))
    return obj


def build(verbose: bool = False, jobs: int | None = None) -> str:
    """Compile every source and link libgdr.so; always rebuilds."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), max(1, (os.cpu_count() or 2)))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc(), "-shared", "-fPIC", "--offload-arch=" + ARCH, "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr[-4000:]))
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
