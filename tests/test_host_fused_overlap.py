"""Outputs of the fused and gated products that share memory with another
output or an operand are refused (CPU only: fake addresses, no kernel launch)."""
import os
import random

import pytest
import torch

from tests.test_host_fused import BACK, FUSED, FUSED8, GATED, GATED8, GBACK, call, f  # noqa: F401 (f: fixture)

ARG, UNSUPPORTED = -8, -7
MB = 1 << 20
# Where a call passes every check it ends at the missing device; with one, these addresses would be used.
without_gpu = pytest.mark.skipif(torch.cuda.is_available() or os.path.exists("/dev/kfd"), reason="fake addresses")


def at(i):
    return 0x100000000 + i * MB


SIZES = dict(M=64, N=64, K=64)
CALLS = {
    "fp8_gemm_nt_fused": (FUSED8, dict(A=at(0), lda=64, a=0, B=at(1), ldb=64, b=0, sa=at(2), na=64, sb=at(3), nb=64,
                                       bias=at(4), act=0, R=at(5), ldr=64, D=at(6), ldd=64, **SIZES)),
    "fp8_gated_nt": (GATED8, dict(A=at(0), lda=64, a=0, G=at(1), ldg=64, U=at(2), ldu=64, w=0, sa=at(3), na=64, sg=at(4),
                                  su=at(5), nw=64, act=2, D=at(6), ldd=64, **SIZES)),
    "bf16_gemm_nt_fused": (FUSED, dict(A=at(0), lda=64, B=at(1), ldb=64, bias=at(2), act=1, R=at(3), ldr=64, D=at(4),
                                       ldd=64, pre=at(5), ldp=64, **SIZES)),
    "bf16_gated_nt": (GATED, dict(A=at(0), lda=64, G=at(1), ldg=64, U=at(2), ldu=64, act=2, D=at(3), ldd=64, pg=at(4),
                                  pu=at(5), ldp=64, **SIZES)),
    "bf16_gemm_nt_fused_backward": (BACK, dict(G=at(0), ldg=64, A=at(1), lda=64, B=at(2), ldb=64, pre=at(3), ldp=64,
                                               act=2, dA=at(4), ldda=64, dB=at(5), lddb=64, dbias=at(6), ws=at(7),
                                               bytes=1 << 30, **SIZES)),
    "bf16_gated_nt_backward": (GBACK, dict(dH=at(0), ldh=64, A=at(1), lda=64, G=at(2), ldg=64, U=at(3), ldu=64, pg=at(4),
                                           pu=at(5), ldp=64, act=2, dA=at(6), ldda=64, dG=at(7), dU=at(8), lddw=64,
                                           ws=at(9), bytes=1 << 30, **SIZES)),
}
OUTPUTS = {"fp8_gemm_nt_fused": ("D",), "fp8_gated_nt": ("D",), "bf16_gemm_nt_fused": ("D", "pre"),
           "bf16_gated_nt": ("D", "pg", "pu"), "bf16_gemm_nt_fused_backward": ("dA", "dB", "dbias", "ws"),
           "bf16_gated_nt_backward": ("dA", "dG", "dU", "ws")}
PAIRS = [(name, out, other) for name, (_, args) in CALLS.items() for out in OUTPUTS[name]
         for other, v in args.items() if isinstance(v, int) and v >= at(0) and other != out]


@pytest.mark.parametrize("name,out,other", PAIRS)
def test_shared_memory_is_refused(f, name, out, other):
    order, args = CALLS[name]
    # 256 bytes into the other one (each spans at least 256 bytes, from 64 floats on), or from 256 bytes before it on
    for place in (args[other], args[other] + 256 - 16, args[other] - 256 + 16):
        if out == "ws":
            place = args[other] // 256 * 256
        if (out, other) == ("D", "R") and place == args[other]:
            continue                               # in place
        st, msg = call(f, name, order, args, **{out: place})
        assert st == ARG and "overlap" in msg, msg


@without_gpu
@pytest.mark.parametrize("name", CALLS)
def test_memory_apart_is_accepted(f, name):
    order, args = CALLS[name]
    assert call(f, name, order, args)[0] == UNSUPPORTED


@without_gpu
def test_residual_in_place_is_accepted(f):
    for name in ("fp8_gemm_nt_fused", "bf16_gemm_nt_fused"):
        order, args = CALLS[name]
        assert call(f, name, order, args, R=args["D"])[0] == UNSUPPORTED
        assert call(f, name, order, args, R=args["D"], M=1, ldr=72)[0] == (ARG if "na" in args else UNSUPPORTED)  # (64 scales)
        assert call(f, name, order, args, R=args["D"], ldr=72)[0] == ARG


@without_gpu
def test_against_sets_of_bytes(f):
    """Matrices anywhere in a small span of memory, of equal and of different strides."""
    rng = random.Random(5)
    order, args = CALLS["bf16_gemm_nt_fused"]
    seen = {True: 0, False: 0}
    for _ in range(4000):
        M, N = rng.randint(1, 6), rng.randint(1, 20)
        ldd = rng.choice((24, 32, 48, 64))
        ldr = ldd if rng.random() < 0.6 else rng.randint(N, 70)
        d, r = at(20) + 16 * rng.randint(0, 40), at(20) + 2 * rng.randint(0, 320)
        if d == r and (ldd == ldr or M == 1):
            continue
        D = {d + 2 * (i * ldd + j) for i in range(M) for j in range(N)}
        R = {r + 2 * (i * ldr + j) for i in range(M) for j in range(N)}
        apart = D.isdisjoint(R)
        st, msg = call(f, "bf16_gemm_nt_fused", order, args, M=M, N=N, K=8, D=d, ldd=ldd, R=r, ldr=ldr, pre=None, ldp=0)
        assert st == (UNSUPPORTED if apart else ARG), (M, N, ldd, ldr, d - r, msg)
        seen[apart] += 1
    assert min(seen.values()) > 500
