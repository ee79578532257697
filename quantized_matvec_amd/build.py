"""Builds libqmv.so in-tree with hipcc for gfx950.

    python -m quantized_matvec_amd.build

Each HIP source is compiled to an object under ``_build/`` (in parallel) and
the objects are linked into ``quantized_matvec_amd/libqmv.so``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqmv.so")
SOURCES = ["qmv_api.hip", "qmv_codec.hip", "qmv_blockwise.hip", "qmv_embedding.hip", "qmv_gemv.hip",
           "qmv_gemm.hip", "qmv_probe.hip", "qmv_rotary.hip", "qmv_kv.hip", "qmv_attention.hip",
           "qmv_attention_decode.hip", "qmv_attention_prompt.hip", "qmv_attention_api.hip", "qmv_lora.hip",
           "qmv_loss.hip", "qmv_decode_piece.hip", "qmv_skinny.hip",
           "qmv_tuning_api.hip"]
ARCH = "gfx950"

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-Wno-unused-function",
    # no implicit multiply-add fusion anywhere: the codec's results are defined
    # with separate roundings; kernels that want an FMA call fmaf() explicitly
    "-ffp-contract=off",
    # packed-fp32 instructions are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES), int(os.environ.get("MAX_JOBS", "8")), 16)
    with ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
