"""Build the gfx950 HIP library in-tree: fp8_gemm_amd/libfp8gemm.so."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SRC = os.path.join(CSRC, "fp8_gemm.hip")           # the plain, block-scaled, per-channel and grouped forms
EXPERTS_SRCS = [os.path.join(CSRC, f) for f in ("experts_bf16.hip", "experts_int8.hip")]
# every unit on the bodies with fused epilogues
FUSED_SRCS = [os.path.join(CSRC, f) for f in ("fused_fp8.hip", "fused_bf16.hip")] + EXPERTS_SRCS
DEPS = [os.path.join(CSRC, f) for f in ("kernels.hpp", "device_common.hpp", "ragged.hpp", "fused.hpp", "tile_halves.hpp",
                                        "fused_bf16.hpp", "fused_host.hpp", "experts.hpp", "experts_host.hpp", "quantize.hpp",
                                        "host_common.hpp")] + \
       [os.path.join(ROOT, "include", f) for f in ("fp8_gemm.h", "fp8_gemm_fused.h", "fp8_gemm_experts.h")]
LIB = os.path.join(HERE, "libfp8gemm.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # no packed FP32 VALU ops (v_pk_add/mul/fma_f32) anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(force: bool = True) -> str:
    """Compile the library (its translation units side by side).  Always recompiles when force is True."""
    srcs = [SRC] + FUSED_SRCS
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(p) for p in srcs + DEPS)
        if os.path.getmtime(LIB) >= newest:
            return LIB
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(s) + ".o") for s in srcs]
        flags = [f for f in HIPCC_FLAGS if f != "-shared"]

        def compile_one(src, obj):
            subprocess.run([hipcc()] + flags + ["-c", src, "-o", obj], check=True)

        with ThreadPoolExecutor(len(srcs)) as pool:
            list(pool.map(compile_one, srcs, objs))
        out = LIB + ".tmp"
        subprocess.run([hipcc()] + HIPCC_FLAGS + objs + ["-o", out], check=True)
        os.replace(out, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
