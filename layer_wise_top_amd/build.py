"""Build the gfx950 shared library liblags.so in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "liblags.so")
SOURCES = [os.path.join(CSRC, "lags_host.cpp"), os.path.join(CSRC, "lags_schedule.cpp"),
           os.path.join(CSRC, "lags_kernels.hip"), os.path.join(CSRC, "lags_act.cpp"),
           os.path.join(CSRC, "lags_ckpt.hip"), os.path.join(CSRC, "lags_gn.hip"),
           os.path.join(CSRC, "lags_gn_f32.hip"), os.path.join(CSRC, "lags_gn_bf16.hip"),
           os.path.join(CSRC, "lags_gn_f16.hip"),
           os.path.join(CSRC, "lags_wgrad.hip")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # no FMA contraction anywhere: the update is a rounded product, then a subtraction
    "-ffp-contract=off",
    # no packed fp32 instructions (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
    "-parallel-jobs=8",
]


def build(verbose: bool = False) -> str:
    cmd = [HIPCC, *FLAGS, "-I", INCLUDE, "-I", CSRC, *SOURCES, "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        sys.stderr.write(proc.stdout + proc.stderr)
        raise RuntimeError("hipcc failed building liblags.so")
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
