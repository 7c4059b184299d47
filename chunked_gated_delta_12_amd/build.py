"""Build libkda.so (HIP for gfx950) in-tree with hipcc.

    python -m chunked_gated_delta_12_amd.build

Each translation unit is compiled on its own (in parallel) and then linked into
chunked_gated_delta_12_amd/libkda.so.  The reference measurements of
include/kda_peaks.h (a streaming copy, a bf16 matrix-core loop, the device's
description) go into a library of their own, libkda_peaks.so.  Packed fp32
instructions are disabled for all device code.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkda.so")
PEAKS_LIB = os.path.join(HERE, "libkda_peaks.so")
PEAKS_SOURCES = ["kda_peaks.hip"]
SOURCES = ["kda_api.cpp", "kda_gate.hip", "kda_decode.hip", "kda_chunk.hip", "kda_map.hip", "kda_out.hip", "kda_bwd.hip", "kda_bwd2.hip", "kda_gmap.hip"]
# the operators beside KDA (the gated delta rule with one decay a head, the norms, the
# selective scan, the short convolution), linked into libkda.so with the sources above
MORE_SOURCES = ["kda_gdr_step.hip", "kda_gdr_chunk.hip", "kda_gdr_prep.hip", "kda_gdr_chain.hip", "kda_gdr_grad.hip",
                "kda_norm.hip", "kda_layer_norm.hip", "kda_conv.hip", "kda_scan_fwd.hip", "kda_scan_bwd.hip", "kda_scan_step.hip"]
ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build libkda)")


def _flags():
    return ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-function", "-I", os.path.join(HERE, "..", "include")]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, src + ".o")
    cmd = [hipcc()] + _flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{res.stderr}")
    return obj


def _link(objs, lib):
    tmp = lib + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(lib)} failed:\n{res.stderr}")
    os.replace(tmp, lib)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = SOURCES + MORE_SOURCES + PEAKS_SOURCES
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = dict(zip(srcs, ex.map(_compile, srcs)))
    _link([objs[s] for s in SOURCES + MORE_SOURCES], LIB)
    _link([objs[s] for s in PEAKS_SOURCES], PEAKS_LIB)
    if verbose:
        print(f"built {LIB} and {PEAKS_LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
