"""Host-side checks of the experts' and integer entry points (CPU only: invalid
arguments or nothing to launch, fake addresses, no kernel launch)."""
import ctypes

import pytest
import torch

from tests.test_host_fused import call, f  # noqa: F401 (f: fixture)
from tests.test_host_fused_overlap import ARG, UNSUPPORTED, at, without_gpu

SIZES = dict(M=64, G=4, N=64, K=64)
FWD = "A lda B ldb step off D ldd M G N K"
BWD = "dD ldg A lda B ldb step off dA ldda dB lddb dstep M G N K"
FWD8 = "A lda B ldb step sa sb off D ldd M G N K"
DENSE8 = "A lda B ldb sa na sb nb bias act R ldr D ldd M N K"
QUANT = "X ldx Q ldq s M K"
CALLS = {
    "bf16_grouped_gemm_ragged": (FWD, dict(A=at(0), lda=64, B=at(1), ldb=64, step=4096, off=at(2), D=at(3), ldd=64, **SIZES)),
    "bf16_grouped_gemm_ragged_backward": (BWD, dict(dD=at(0), ldg=64, A=at(1), lda=64, B=at(2), ldb=64, step=4096, off=at(3),
                                                    dA=at(4), ldda=64, dB=at(5), lddb=64, dstep=4096, **SIZES)),
    "int8_grouped_gemm_ragged": (FWD8, dict(A=at(0), lda=64, B=at(1), ldb=64, step=4096, sa=at(2), sb=at(3), off=at(4),
                                            D=at(5), ldd=64, **SIZES)),
    "int8_gemm_nt_fused": (DENSE8, dict(A=at(0), lda=64, B=at(1), ldb=64, sa=at(2), na=64, sb=at(3), nb=64, bias=at(4), act=0,
                                        R=at(5), ldr=64, D=at(6), ldd=64, M=64, N=64, K=64)),
    "int8_quantize_rows": (QUANT, dict(X=at(0), ldx=64, Q=at(1), ldq=64, s=at(2), M=64, K=64)),
}
OUTPUTS = {"bf16_grouped_gemm_ragged": ("D",), "bf16_grouped_gemm_ragged_backward": ("dA", "dB"),
           "int8_grouped_gemm_ragged": ("D",), "int8_gemm_nt_fused": ("D",), "int8_quantize_rows": ("Q", "s")}


def refused(f, name, status, **kw):  # noqa: F811
    st, msg = call(f, name, *CALLS[name], **kw)
    assert st == status and ":" in msg, (st, msg)
    return msg


@pytest.mark.parametrize("name", ["bf16_grouped_gemm_ragged", "int8_grouped_gemm_ragged"])
@pytest.mark.parametrize("kw,status", [
    (dict(A=None), -1), (dict(B=None), -1), (dict(D=None), -1), (dict(off=None), -1),
    (dict(A=at(0) + 8), -3), (dict(B=at(1) + 2), -3), (dict(D=at(3) + 8), -3), (dict(off=at(2) + 2), -3),
    (dict(lda=68), -3), (dict(ldd=68), -3), (dict(step=4100), -3),
    (dict(lda=48), -5), (dict(ldb=1 << 24), -5), (dict(ldd=56), -5), (dict(step=4080), -5), (dict(step=0), -5), (dict(step=-4096), -5),
    (dict(K=20), -2), (dict(N=60), -2), (dict(M=-1), -2), (dict(G=-1), -2), (dict(G=65536), -2), (dict(N=1 << 23), -2), (dict(K=1 << 23), -2),
])
def test_ragged_refusals(f, name, kw, status):  # noqa: F811
    refused(f, name, status, **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(dD=None), -1), (dict(A=None), -1), (dict(B=None), -1), (dict(off=None), -1),
    (dict(dD=at(0) + 2), -3), (dict(ldg=68), -3), (dict(ldg=56), -5), (dict(ldda=56), -5), (dict(dA=at(4) + 8), -3),
    (dict(lddb=60), -5), (dict(dstep=4080), -5), (dict(dstep=4100), -3), (dict(step=64), -5), (dict(K=12), -2), (dict(N=12), -2),
    (dict(M=(1 << 30) + 1), -2),
])
def test_backward_refusals(f, kw, status):  # noqa: F811
    refused(f, "bf16_grouped_gemm_ragged_backward", status, **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(A=None), -1), (dict(B=None), -1), (dict(D=None), -1), (dict(lda=72), -3), (dict(R=at(5) + 1), -3), (dict(ldr=60), -5),
    (dict(sa=at(2) + 2), -3), (dict(na=3), -8), (dict(nb=65), -8), (dict(act=5), -8), (dict(act=-1), -8), (dict(K=24), -2),
    (dict(K=131072, lda=131072, ldb=131072), -2), (dict(M=-1), -2),
])
def test_int8_refusals(f, kw, status):  # noqa: F811
    refused(f, "int8_gemm_nt_fused", status, **kw)


def test_int8_longest_sum(f):  # noqa: F811
    """131056 products of -128 by -128 stay below 2^31, 131072 do not."""
    assert 131056 * 2 ** 14 < 2 ** 31 <= 131072 * 2 ** 14
    msg = refused(f, "int8_grouped_gemm_ragged", -2, K=131072, lda=131072, ldb=131072, step=64 * 131072)
    assert "131056" in msg


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), -1), (dict(Q=None), -1), (dict(s=None), -1), (dict(X=at(0) + 2), -3), (dict(Q=at(1) + 8), -3),
    (dict(s=at(2) + 2), -3), (dict(ldx=68), -3), (dict(ldx=56), -5), (dict(ldq=48), -5), (dict(ldq=72), -3), (dict(K=24), -2),
    (dict(K=-16), -2), (dict(M=-1), -2),
])
def test_quantise_refusals(f, kw, status):  # noqa: F811
    refused(f, "int8_quantize_rows", status, **kw)


PAIRS = [(name, out, other) for name, (_, args) in CALLS.items() for out in OUTPUTS[name]
         for other, v in args.items() if isinstance(v, int) and v >= at(0) and other != out and other != "off"]


@pytest.mark.parametrize("name,out,other", PAIRS)
def test_shared_memory_is_refused(f, name, out, other):  # noqa: F811
    args = CALLS[name][1]
    for place in (args[other], args[other] + 256 - 16, args[other] - 256 + 16):
        if (out, other) == ("D", "R") and place == args[other]:
            continue                               # in place
        assert "overlap" in refused(f, name, ARG, **{out: place})


def test_every_experts_memory_counts(f):  # noqa: F811
    """An output inside the last expert's weights, or over the offsets."""
    name = "bf16_grouped_gemm_ragged"
    for step in (4096, 8192):                      # one matrix behind the other, and apart
        last = CALLS[name][1]["B"] + 2 * 3 * step
        assert "overlap" in refused(f, name, ARG, step=step, D=last + 8192 - 16)
    assert "overlap" in refused(f, name, ARG, D=at(2) + 16 - 8192 + 16 - 16)
    assert "overlap" in refused(f, "bf16_grouped_gemm_ragged_backward", ARG, dB=at(3) - 4 * 8192 + 16)


@without_gpu
@pytest.mark.parametrize("name", CALLS)
def test_memory_apart_is_accepted(f, name):  # noqa: F811
    st, msg = call(f, name, *CALLS[name])
    assert st == UNSUPPORTED, msg


@without_gpu
def test_in_place_residual_and_columns(f):  # noqa: F811
    assert call(f, "int8_gemm_nt_fused", *CALLS["int8_gemm_nt_fused"], R=at(6))[0] == UNSUPPORTED
    # the output as the columns behind the operand's, in one buffer
    assert call(f, "bf16_grouped_gemm_ragged", *CALLS["bf16_grouped_gemm_ragged"], lda=128, ldd=128, D=at(0) + 128)[0] == UNSUPPORTED
    # weights as halves of a merged [G, 2 N, K] matrix
    assert call(f, "bf16_grouped_gemm_ragged", *CALLS["bf16_grouped_gemm_ragged"], step=8192)[0] == UNSUPPORTED


def test_nothing_to_launch(f):  # noqa: F811
    for name in ("bf16_grouped_gemm_ragged", "int8_grouped_gemm_ragged"):
        for kw in (dict(M=0), dict(G=0), dict(N=0)):
            assert call(f, name, *CALLS[name], **kw)[0] == 0
    assert call(f, "int8_gemm_nt_fused", *CALLS["int8_gemm_nt_fused"], M=0)[0] == 0
    assert call(f, "int8_gemm_nt_fused", *CALLS["int8_gemm_nt_fused"], N=0)[0] == 0
    assert call(f, "int8_quantize_rows", *CALLS["int8_quantize_rows"], M=0)[0] == 0
    assert call(f, "bf16_grouped_gemm_ragged_backward", *CALLS["bf16_grouped_gemm_ragged_backward"], dA=None, dB=None)[0] == 0
    assert call(f, "bf16_grouped_gemm_ragged_backward", *CALLS["bf16_grouped_gemm_ragged_backward"], M=0, dB=None)[0] == 0
    assert call(f, "bf16_grouped_gemm_ragged_backward", *CALLS["bf16_grouped_gemm_ragged_backward"], K=0)[0] == 0


@pytest.mark.parametrize("op,m,n,k,g,variant", [
    (0, 8, 2048, 4096, 64, 4), (0, 640, 2048, 4096, 64, 4), (0, 8192, 14336, 4096, 8, 1), (1, 512, 2048, 7168, 64, 4),
    (1, 65536, 2048, 4096, 64, 1), (2, 8192, 14336, 4096, 8, 1), (3, 8192, 14336, 4096, 8, 1), (4, 1, 4096, 4096, 1, 4),
    (4, 8192, 8192, 4096, 1, 1), (0, 0, 8, 8, 1, 0), (2, 5, 8, 0, 1, 0), (3, 5, 8, 8, 0, 0), (2, 5, 8, 8, 0, 7), (3, 0, 8, 8, 2, 7),
])
def test_plan(f, op, m, n, k, g, variant):  # noqa: F811
    p = f.experts_plan(op, m, n, k, g)
    assert p.variant == variant
    if variant and op < 3:
        # as many row tiles as any offsets can need: every expert (and, for op 2, the rows of none) may start one
        live = min(g + (2 if op == 2 else 0), m)
        cols = k if op == 2 else n
        assert p.workgroups == (m + live * (p.tile_m - 1)) // p.tile_m * -(-cols // p.tile_n)


def test_tiles_of_any_offsets_fit_the_launch(f):  # noqa: F811
    import random
    rng = random.Random(3)
    for _ in range(300):
        g, m = rng.randint(1, 9), rng.randint(1, 900)
        for op, k in ((0, 64), (1, 64), (2, 2048)):
            p = f.experts_plan(op, m, 64, k, g)
            cuts = sorted(rng.randint(0, m) for _ in range(g + 1))
            bounds = [0] + cuts + [m] if op == 2 else cuts
            tiles = sum(-(-(b - a) // p.tile_m) for a, b in zip(bounds, bounds[1:]))
            assert tiles * -(-(k if op == 2 else 64) // p.tile_n) <= p.workgroups


def test_plan_refusals(f):  # noqa: F811
    for args, status in (((5, 1, 8, 16, 1), -8), ((-1, 1, 8, 16, 1), -8), ((0, 1, 8, 12, 1), -2), ((0, 1, 9, 8, 1), -2), ((0, 1, 8, 8, -1), -2)):
        with pytest.raises(f.Fp8GemmError) as e:
            f.experts_plan(*args)
        assert e.value.status == status
    assert f.load_library().fp8_gemm_experts_plan(0, 1, 8, 8, 1, None) == -1
    plan = f.Plan()
    for op in range(5):
        for m in (1, 16, 65, 100000, (1 << 31) - 1):
            for n in (8, 136, 28672, 1 << 21):
                for k in (0, 16, 1 << 20):
                    for g in (1, 64, 65535):
                        assert f.load_library().fp8_gemm_experts_plan(op, m, n, k, g, ctypes.byref(plan)) == 0
                        assert plan.variant in (0, 1, 2, 4, 7)


def test_wrapper_refusals(f):  # noqa: F811
    bf = torch.bfloat16
    a, b, o = torch.zeros(4, 32, dtype=bf), torch.zeros(2, 8, 32, dtype=bf), torch.zeros(3, dtype=torch.int32)
    a8, b8 = a.to(torch.int8), b.to(torch.int8)
    with pytest.raises(ValueError, match="GPU"):
        f.grouped_gemm_ragged_bf16(a, b, o)
    with pytest.raises(ValueError, match="GPU"):
        f.grouped_gemm_ragged_int8(a8, b8, o)
    with pytest.raises(ValueError, match="GPU"):
        f.quantize_rows_int8(a)
    with pytest.raises(ValueError, match="GPU"):
        f.gemm_nt_int8(a8, b8[0])
    with pytest.raises(TypeError):
        f.grouped_gemm_ragged_bf16(a.float(), b, o)
    with pytest.raises(TypeError):
        f.gemm_nt_int8(a8.view(torch.uint8), b8[0])
    with pytest.raises(TypeError):
        f.quantize_rows_int8(a.float())
    with pytest.raises(ValueError, match="not .M, K."):
        f.grouped_gemm_ragged_bf16(a, b[0], o)
    with pytest.raises(ValueError, match="offsets"):
        f.grouped_gemm_ragged_bf16(a, b, o[:2])
    with pytest.raises(ValueError, match="offsets"):
        f.grouped_gemm_ragged_bf16(a, b, o.long())
    with pytest.raises(ValueError, match="grad_out"):
        f.grouped_gemm_ragged_bf16_backward(torch.zeros(4, 9, dtype=bf), a, b, o)
    with pytest.raises(ValueError, match="K-contiguous"):
        f._expert_weights(torch.zeros(2, 32, 8).transpose(1, 2), 2, 8, 32, 8)
    with pytest.raises(ValueError, match="x must be"):
        f.quantize_rows_int8(b)
