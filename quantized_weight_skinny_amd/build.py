"""Build libqpn.so (the HIP kernels and the C ABI of include/qpn.h,
include/qpn_decode.h and include/qpn_prompt.h) for gfx950.

Run ``python -m quantized_weight_skinny_amd.build`` (or call ``build()``); the
library lands next to this file so that it travels with the source tree.
"""

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["qpn_api.hip", "qpn_gemm.hip", "qpn_mlp.hip", "qpn_pack.hip", "qpn_plan.cpp", "qpn_checks.cpp",
           "qpn_decode_api.hip", "qpn_kv4_attention.hip", "qpn_kv4_cache.hip", "qpn_verify.hip",
           "qpn_decode_checks.cpp", "qpn_prompt_api.hip", "qpn_fp8_block.hip", "qpn_kv4_chunk.hip", "qpn_logprobs.hip",
           "qpn_prompt_checks.cpp"]
LIB = os.path.join(HERE, "libqpn.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    "-parallel-jobs=8",
    # keep the compiler from forming packed fp32 (v_pk_*_f32) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def build(verbose=False):
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB + ".tmp"
    cmd = [HIPCC, *FLAGS, *srcs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed with exit code {res.returncode}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
