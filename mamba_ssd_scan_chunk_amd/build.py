"""Build the gfx950 HIP library ``libmamba_ssd.so`` in-tree with hipcc.

Usage: ``python -m mamba_ssd_scan_chunk_amd.build`` (or ``build()``).
Every translation unit is compiled for gfx950 only, in parallel, then linked
into one shared library next to this file.
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
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libmamba_ssd.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)

SOURCES = ["chunk_cumsum.hip", "chunk_state.hip", "chunk_state_hg.hip", "state_passing.hip", "state_fused.hip", "forward_fused.hip",
           "chunk_scan.hip", "chunk_scan_hg.hip", "decode.hip", "varlen_states.hip", "backward.hip", "bwd_dbc.hip",
           "ssd_api.cpp", "tuning.cpp", "forward_noalloc.hip", "causal_conv.hip", "selective_scan.hip",
           "selective_scan_bwd.hip", "layer_norm.hip", "layer_api.cpp", "delta_rule.hip", "delta_rule_bwd.hip",
           "delta_api.cpp", "group_norm.hip", "group_api.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17", "-Wall",
    # packed-fp32 vector ops off: ordinary scalar/float2 code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "not a recognized feature for this target"
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msgs}")
    if msgs.strip():
        print(msgs, file=sys.stderr)
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
