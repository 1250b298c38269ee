"""Host-side checks of the fused and gated entry points (CPU only, no kernel launch).

Argument sets are invalid, or leave nothing to launch: validation ends before
any pointer is used.  The Python wrappers' own checks are made on CPU tensors.
"""
import ctypes
import os

import pytest
import torch

A16, A256, ODD2 = 0x10000, 0x20000, 0x10002     # fake addresses (never dereferenced)


@pytest.fixture(scope="module")
def f():
    import fp8_gemm_amd
    from fp8_gemm_amd import _build
    if not os.path.exists(fp8_gemm_amd.LIB_PATH):
        _build.build()
    fp8_gemm_amd.load_library()
    return fp8_gemm_amd


def call(f, name, order, base, **kw):
    args = dict(base)
    args.update(kw)
    lib = f.load_library()
    st = getattr(lib, name)(*(args[k] for k in order.split()), None)
    return st, lib.fp8_gemm_strerror(st).decode()


FUSED8 = "A lda a B ldb b sa na sb nb bias act R ldr D ldd M N K"
FUSED8_OK = dict(A=A16, lda=128, a=0, B=A16, ldb=128, b=0, sa=A16, na=128, sb=A16, nb=128, bias=A16, act=0, R=A16, ldr=128,
                 D=A16, ldd=128, M=128, N=128, K=128)


@pytest.mark.parametrize("kw,status", [
    (dict(A=None), -1), (dict(B=None), -1), (dict(D=None), -1),
    (dict(A=0x10008), -3), (dict(D=0x10008), -3), (dict(lda=136), -3), (dict(ldd=132), -3), (dict(sa=ODD2), -3),
    (dict(sb=ODD2), -3), (dict(bias=ODD2), -3), (dict(R=0x10001), -3),
    (dict(a=2), -4), (dict(b=-1), -4),
    (dict(lda=112), -5), (dict(ldb=1 << 24), -5), (dict(ldd=120), -5), (dict(ldr=127), -5),
    (dict(K=24), -2), (dict(M=-1), -2), (dict(N=-1), -2), (dict(K=1 << 23), -2),
    (dict(act=5), -8), (dict(act=-1), -8), (dict(na=2), -8), (dict(nb=127), -8),
])
def test_fused_fp8_refusals(f, kw, status):
    st, msg = call(f, "fp8_gemm_nt_fused", FUSED8, FUSED8_OK, **kw)
    assert st == status and ":" in msg, msg


GATED8 = "A lda a G ldg U ldu w sa na sg su nw act D ldd M N K"
GATED8_OK = dict(A=A16, lda=128, a=0, G=A16, ldg=128, U=A16, ldu=256, w=0, sa=A16, na=1, sg=A16, su=A16, nw=128, act=2,
                 D=A16, ldd=128, M=128, N=128, K=128)


@pytest.mark.parametrize("kw,status", [
    (dict(A=None), -1), (dict(G=None), -1), (dict(U=None), -1), (dict(D=None), -1),
    (dict(U=0x10008), -3), (dict(ldu=136), -3), (dict(ldu=112), -5), (dict(ldg=112), -5), (dict(w=2), -4),
    (dict(nw=3), -8), (dict(act=9), -8), (dict(K=8), -2), (dict(su=ODD2), -3),
])
def test_gated_fp8_refusals(f, kw, status):
    st, msg = call(f, "fp8_gated_nt", GATED8, GATED8_OK, **kw)
    assert st == status and ":" in msg, msg


FUSED = "A lda B ldb bias act R ldr D ldd pre ldp M N K"
FUSED_OK = dict(A=A16, lda=128, B=A16, ldb=128, bias=None, act=1, R=None, ldr=0, D=A16, ldd=128, pre=None, ldp=0, M=128,
                N=128, K=128)


@pytest.mark.parametrize("kw,status", [
    (dict(A=None), -1), (dict(D=None), -1), (dict(A=0x10008), -3), (dict(lda=132), -3), (dict(lda=120), -5),
    (dict(lda=1 << 22), -5), (dict(K=12), -2), (dict(pre=ODD2, ldp=128), -3), (dict(pre=A16, ldp=127), -5), (dict(act=7), -8),
])
def test_fused_bf16_refusals(f, kw, status):
    st, msg = call(f, "bf16_gemm_nt_fused", FUSED, FUSED_OK, **kw)
    assert st == status and ":" in msg, msg


GATED = "A lda G ldg U ldu act D ldd pg pu ldp M N K"
GATED_OK = dict(A=A16, lda=128, G=A16, ldg=128, U=A16, ldu=128, act=2, D=A16, ldd=128, pg=A16, pu=A16, ldp=128, M=128, N=128,
                K=128)


@pytest.mark.parametrize("kw,status", [
    (dict(G=None), -1), (dict(pg=None), -1), (dict(pu=None), -1), (dict(ldp=100), -5), (dict(pu=ODD2), -3), (dict(K=4), -2),
])
def test_gated_bf16_refusals(f, kw, status):
    st, msg = call(f, "bf16_gated_nt", GATED, GATED_OK, **kw)
    assert st == status and ":" in msg, msg


BACK = "G ldg A lda B ldb pre ldp act dA ldda dB lddb dbias ws bytes M N K"
BACK_OK = dict(G=A16, ldg=128, A=A16, lda=128, B=A16, ldb=128, pre=A16, ldp=128, act=2, dA=A16, ldda=128, dB=A16, lddb=128,
               dbias=A16, ws=A256, bytes=1 << 30, M=128, N=128, K=128)


@pytest.mark.parametrize("kw,status", [
    (dict(G=None), -1), (dict(A=None), -1), (dict(B=None), -1), (dict(pre=None), -1), (dict(ws=None), -1),
    (dict(ws=0x20080), -3), (dict(bytes=1000), -8), (dict(ldg=100), -5), (dict(ldda=100), -5), (dict(lddb=132), -3),
    (dict(dA=0x10008), -3), (dict(dbias=ODD2), -3), (dict(G=0x10001), -3), (dict(act=8), -8), (dict(K=12), -2),
    (dict(M=(1 << 30) + 1), -2), (dict(N=1 << 22), -2),
])
def test_fused_backward_refusals(f, kw, status):
    st, msg = call(f, "bf16_gemm_nt_fused_backward", BACK, BACK_OK, **kw)
    assert st == status and ":" in msg, msg


GBACK = "dH ldh A lda G ldg U ldu pg pu ldp act dA ldda dG dU lddw ws bytes M N K"
GBACK_OK = dict(dH=A16, ldh=128, A=A16, lda=128, G=A16, ldg=128, U=A16, ldu=128, pg=A16, pu=A16, ldp=128, act=2, dA=A16,
                ldda=128, dG=A16, dU=A16, lddw=128, ws=A256, bytes=1 << 30, M=128, N=128, K=128)


@pytest.mark.parametrize("kw,status", [
    (dict(dH=None), -1), (dict(pg=None), -1), (dict(dG=None), -1), (dict(dU=None), -1), (dict(A=None), -1), (dict(U=None), -1),
    (dict(ldu=136), -5), (dict(bytes=100), -8), (dict(ws=0x20010), -3), (dict(ldh=127), -5),
])
def test_gated_backward_refusals(f, kw, status):
    st, msg = call(f, "bf16_gated_nt_backward", GBACK, GBACK_OK, **kw)
    assert st == status and ":" in msg, msg


def test_nothing_to_launch(f):
    for name, order, base in (("fp8_gemm_nt_fused", FUSED8, FUSED8_OK), ("fp8_gated_nt", GATED8, GATED8_OK),
                              ("bf16_gemm_nt_fused", FUSED, FUSED_OK), ("bf16_gated_nt", GATED, GATED_OK)):
        assert call(f, name, order, base, M=0)[0] == 0 and call(f, name, order, base, N=0)[0] == 0
    assert call(f, "bf16_gemm_nt_fused_backward", BACK, BACK_OK, M=0, N=0)[0] == 0
    assert call(f, "bf16_gated_nt_backward", GBACK, GBACK_OK, dA=None, dG=None, dU=None)[0] == 0
    assert call(f, "bf16_gated_nt_backward", GBACK, GBACK_OK, K=0)[0] == 0


def test_workspaces(f):
    lib = f.load_library()
    for M, N, K in ((0, 0, 0), (1, 1, 8), (64, 64, 64), (65, 129, 1000), (5, 14336, 4096), (8192, 128, 128), (4096, 14336, 4096)):
        cols = (N + 63) // 64 * 64
        # the gradients, the bias sums, and what the split products need
        sums = [0]
        if K:
            for m, k in ((M, cols), (N, M)):
                splits = f.fused_plan(4, m, K, k).k_splits
                sums.append(4 * splits * m * K if splits > 1 else 0)
        need = 2 * M * cols + 4 * ((M + 63) // 64) * N + max(sums)
        assert lib.bf16_gemm_nt_fused_backward_workspace(M, N, K) >= need
        assert lib.bf16_gated_nt_backward_workspace(M, N, K) >= 4 * M * cols
    assert lib.bf16_gated_nt_backward_workspace(-1, 4, 8) == -2
    assert lib.bf16_gemm_nt_fused_backward_workspace(4, 1 << 22, 8) == -2
    assert lib.bf16_gemm_nt_fused_backward_workspace(4, 4, 4) == -2


@pytest.mark.parametrize("m,n,k,splits", [(4096, 4096, 4096, False), (5, 1000, 14336, True), (128, 128, 8192, True),
                                          (1024, 1024, 65536, True), (64, 64, 64, False), (24, 712, 962, True)])
def test_backward_splits(f, m, n, k, splits):
    p = f.fused_plan(4, m, n, k)
    assert (p.k_splits > 1) == splits
    assert p.workgroups == -(-m // p.tile_m) * -(-n // p.tile_n) * p.k_splits
    assert p.k_splits <= 64 and 4 * p.k_splits * m * n <= 128 << 20


@pytest.mark.parametrize("op,m,n,k,variant", [
    (0, 1, 4096, 4096, 4), (0, 64, 4096, 14336, 4), (0, 512, 4096, 4096, 4), (0, 2049, 512, 512, 7), (0, 2048, 4096, 4096, 2), (0, 4096, 4096, 4096, 1),
    (1, 1, 14336, 4096, 4), (1, 64, 14336, 4096, 4), (1, 256, 14336, 4096, 2), (1, 8192, 14336, 4096, 1), (2, 16, 4096, 2048, 4), (3, 4096, 14336, 4096, 1),
    (4, 4096, 4096, 28672, 1), (4, 1, 64, 64, 7), (0, 0, 5, 16, 0), (4, 5, 0, 3, 0),
])
def test_plan(f, op, m, n, k, variant):
    p = f.fused_plan(op, m, n, k)
    assert p.variant == variant
    if variant == 4:
        assert p.workgroups == -(-n // p.tile_n) * -(-m // 64)
    elif variant:
        assert p.workgroups == -(-m // p.tile_m) * -(-n // p.tile_n) * p.k_splits


@pytest.mark.parametrize("op,m,n,k,status", [(5, 1, 1, 16, -8), (-1, 1, 1, 16, -8), (0, 1, 1, 8, -2), (2, 1, 1, 4, -2), (0, -1, 1, 16, -2)])
def test_plan_refusals(f, op, m, n, k, status):
    with pytest.raises(f.Fp8GemmError) as e:
        f.fused_plan(op, m, n, k)
    assert e.value.status == status
    assert f.load_library().fp8_gemm_fused_plan(0, 1, 1, 16, None) == -1


def test_plan_never_faults(f):
    plan = f.Plan()
    lib = f.load_library()
    for op in range(5):
        for m in (1, 16, 17, 64, 65, 512, 513, 100000, (1 << 31) - 1):
            for n in (1, 15, 16, 129, 28672, (1 << 31) - 1):
                for k in (0, 16, 1 << 20):
                    assert lib.fp8_gemm_fused_plan(op, m, n, k, ctypes.byref(plan)) == 0
                    assert plan.variant in (1, 2, 4, 7) and plan.workgroups > 0


def test_wrapper_refusals(f):
    """What the wrappers refuse before the library sees it (here: before a GPU is needed)."""
    bf, e4 = torch.bfloat16, torch.float8_e4m3fn
    a, b = torch.zeros(4, 32, dtype=bf), torch.zeros(8, 32, dtype=bf)
    a8, b8 = torch.zeros(4, 32).to(e4), torch.zeros(8, 32).to(e4)
    with pytest.raises(ValueError, match="GPU"):
        f.gemm_nt_bf16_fused(a, b)
    with pytest.raises(ValueError, match="GPU"):
        f.gemm_nt_fused(a8, b8)
    with pytest.raises(ValueError, match="not .M, K."):
        f.gated_nt_bf16(a, torch.zeros(8, 16, dtype=bf), b)
    with pytest.raises(ValueError, match="w_up"):
        f.gated_nt_bf16(a, b, torch.zeros(9, 32, dtype=bf))
    with pytest.raises(TypeError):
        f.gemm_nt_bf16_fused(a.float(), b)
    with pytest.raises(TypeError):
        f.gemm_nt_fused(a, b)
    with pytest.raises(TypeError):
        f.gemm_nt_fused(a8.view(torch.uint8), b8)
    with pytest.raises(TypeError, match="one FP8 dtype"):
        f.gated_nt(a8, b8, b8.float().to(torch.float8_e5m2))
    with pytest.raises(ValueError, match="activation"):
        f._activation("swish")
    with pytest.raises(ValueError, match="K-contiguous"):
        f._operand(torch.zeros(32, 4).t(), "a", 4, 32, 8)
    with pytest.raises(ValueError, match="row stride"):
        f._rows(torch.zeros(1, 8).expand(4, 8), "residual", 4, 8, torch.float32)
    with pytest.raises(ValueError, match="preact"):
        f._gated_preact(f._tt(), torch.zeros(4, 8), 4, 8)
    with pytest.raises(ValueError, match="1"):
        f._floats(f._tt(), torch.zeros(3), "scale_a", 4)


@pytest.mark.parametrize("M,N,strides,overlap", [
    (4, 8, (32, 8, 1), False), (4, 8, (8, 16, 1), False), (4, 8, (28, 8, 1), True), (4, 8, (0, 8, 1), True),
    (4, 8, (4, 16, 1), True), (4, 8, (8, 12, 1), True), (1, 8, (8, 8, 1), False), (1, 8, (7, 8, 1), True),
    (0, 8, (0, 8, 1), False), (4, 5, (8, 16, 1), False),
])
def test_preact_matrices_overlap(f, M, N, strides, overlap):
    t = torch.zeros(256).as_strided((2, M, N), strides)
    assert overlap == (len(set((r * strides[1] + p * strides[0] + c) for p in range(2) for r in range(M)
                               for c in range(N))) < 2 * M * N)
    if overlap:
        with pytest.raises(ValueError, match="overlap"):
            f._gated_preact(f._tt(), t, M, N)
    else:
        gate, up, ld = f._gated_preact(f._tt(), t, M, N)
        assert up - gate == 4 * strides[0] and ld == (strides[1] if M > 1 else N)


def test_same_matrix_twice(f):
    lib = f.load_library()
    st = lib.bf16_gated_nt(A16, 64, A16, 64, A16, 64, 2, A16, 64, A256, A256, 64, 64, 64, 64, None)
    assert st == -8 and "pre_g and pre_u" in lib.fp8_gemm_strerror(st).decode()
    st = lib.bf16_gated_nt_backward(A16, 64, A16, 64, A16, 64, A16, 64, A16, A16, 64, 2, A16, 64, A256, A256, 64, A256,
                                    1 << 40, 64, 64, 64, None)
    assert st == -8 and "dWg and dWu" in lib.fp8_gemm_strerror(st).decode()
