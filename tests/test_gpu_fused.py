"""GPU parity of the products with a fused epilogue and of the gated products.

References and bounds: tests/_fused.py.  The sizes put every kernel at its
edges: one token, token counts around each class, odd output columns, K tails,
tiles that end inside a matrix.
"""
import itertools

import pytest
import torch

from tests import _fused as F

pytestmark = pytest.mark.gpu

E4, E5, BF = torch.float8_e4m3fn, torch.float8_e5m2, torch.bfloat16
DEV = "cuda:0"


@pytest.fixture(scope="module")
def f():
    import fp8_gemm_amd
    fp8_gemm_amd.load_library()
    return fp8_gemm_amd


def rand(seed, *shape, dtype=BF, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def scales(seed, n):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(n, generator=g) * 1.5 + 0.5).to(DEV)


def strided(t, extra, fill=float("nan")):
    """The same values in rows `extra` elements longer, which hold NaN."""
    big = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=torch.float32).to(t.dtype).to(t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


FP8_SHAPES = [(1, 16, 16), (1, 130, 272), (5, 33, 400), (16, 64, 128), (17, 100, 144), (33, 257, 528), (64, 48, 1040),
              (65, 300, 272), (128, 256, 128), (130, 515, 400), (257, 260, 1168), (300, 1003, 144)]


@pytest.mark.parametrize("M,N,K", FP8_SHAPES)
@pytest.mark.parametrize("kind", [(E4, E4), (E5, E4)], ids=["e4m3", "mixed"])
def test_fused_fp8(f, M, N, K, kind):
    a, b = rand(M + K, M, K, dtype=kind[0]), rand(N + 7 * K, N, K, dtype=kind[1], std=0.25)
    sa, sb = scales(1, M), scales(2, N)
    bias, res = rand(3, N, dtype=torch.float32), rand(4, M, N)
    for i, name in enumerate(F.ACTS):
        args = dict(scale_a=[sa, sa[:1], None][i % 3], scale_b=[sb, None, sb[:1]][i % 3],
                    bias=bias if i % 2 else None, residual=res if i != 2 else None)
        out = f.gemm_nt_fused(a, b, activation=name, **args)
        _, v, tight, hw = F.fused_reference(a, b, args["scale_a"], args["scale_b"], args["bias"], name, args["residual"])
        F.check(out, v, tight, hw, K, f"fused {name} {M}x{N}x{K}")


@pytest.mark.parametrize("fa,fb", itertools.product((E4, E5), (E4, E5)), ids=str)
@pytest.mark.parametrize("M", [7, 40, 200, 600])
def test_fused_fp8_formats(f, M, fa, fb):
    N, K = 320, 320
    a, b = rand(1, M, K, dtype=fa), rand(2, N, K, dtype=fb)
    out = f.gemm_nt_fused(a, b, activation="silu")
    _, v, tight, hw = F.fused_reference(a, b, name="silu")
    F.check(out, v, tight, hw, K, "formats")
    wu = rand(3, N, K, dtype=fb)
    out = f.gated_nt(a, b, wu)
    _, _, v, tight, hw = F.gated_reference(a, b, wu)
    F.check(out, v, tight, hw, K, "gated formats")


@pytest.mark.parametrize("M,N,K", FP8_SHAPES)
@pytest.mark.parametrize("kind", [(E4, E4), (E5, E4)], ids=["e4m3", "mixed"])
def test_gated_fp8(f, M, N, K, kind):
    a = rand(M + K, M, K, dtype=kind[0])
    wg, wu = rand(N + 7 * K, N, K, dtype=kind[1], std=0.25), rand(N + 5 * K, N, K, dtype=kind[1], std=0.25)
    sa, sg, su = scales(1, M), scales(2, N), scales(3, N)
    for i, name in enumerate(F.ACTS):
        args = [(sa, sg, su), (sa[:1], sg[:1], su[:1]), (None, None, su)][i % 3]
        out = f.gated_nt(a, wg, wu, *args, activation=name)
        _, _, v, tight, hw = F.gated_reference(a, wg, wu, *args, name=name)
        F.check(out, v, tight, hw, K, f"gated {name} {M}x{N}x{K}")


BF_SHAPES = [(1, 16, 8), (1, 130, 264), (5, 33, 200), (16, 64, 64), (33, 257, 136), (64, 48, 520), (65, 300, 136),
             (128, 256, 64), (130, 515, 200), (257, 260, 584), (300, 1003, 72)]


@pytest.mark.parametrize("M,N,K", BF_SHAPES)
def test_fused_bf16(f, M, N, K):
    a, b = rand(M + K, M, K), rand(N + 7 * K, N, K, std=0.25)
    bias, res = rand(3, N, dtype=torch.float32), rand(4, M, N)
    for i, name in enumerate(F.ACTS):
        bi, r = (bias if i % 2 else None), (res if i != 2 else None)
        pre = torch.empty((M, N), device=DEV)
        out = f.gemm_nt_bf16_fused(a, b, bias=bi, activation=name, residual=r, preact=pre)
        z, v, tight, hw = F.fused_reference(a, b, bias=bi, name=name, res=r)
        F.check(out, v, tight, hw, K, f"fused {name} {M}x{N}x{K}")
        assert ((pre.cpu().double() - z).abs() <= tight + hw).all()
        assert torch.equal(out, f.gemm_nt_bf16_fused(a, b, bias=bi, activation=name, residual=r))


@pytest.mark.parametrize("M,N,K", BF_SHAPES)
def test_gated_bf16(f, M, N, K):
    a = rand(M + K, M, K)
    wg, wu = rand(N + 7 * K, N, K, std=0.25), rand(N + 5 * K, N, K, std=0.25)
    for name in F.ACTS:
        pre = torch.empty((2, M, N), device=DEV)
        out = f.gated_nt_bf16(a, wg, wu, activation=name, preact=pre)
        g, u, v, tight, hw = F.gated_reference(a, wg, wu, name=name)
        F.check(out, v, tight, hw, K, f"gated {name} {M}x{N}x{K}")
        for p, (z, S, h) in zip(pre, ((g, *F.product(a, wg)[1:]), (u, *F.product(a, wu)[1:]))):
            assert ((p.cpu().double() - z).abs() <= 1e-5 * S + h).all()


def grad_error(name, G, z, zerr):
    e = G.abs() * (0.8 * zerr + 2.0 ** -19 * (1 + z.abs()))
    if name == "relu":
        e = e + torch.where(z.abs() <= zerr, G.abs(), torch.zeros_like(G))
    return e if name != "none" else torch.zeros_like(G)


@pytest.mark.parametrize("M,N,K", BF_SHAPES)
@pytest.mark.parametrize("name", F.ACTS)
def test_fused_bf16_backward(f, M, N, K, name):
    a, b, G = rand(M + K, M, K), rand(N + 7 * K, N, K, std=0.25), rand(9, M, N)
    bias = rand(3, N, dtype=torch.float32)
    pre = torch.empty((M, N), device=DEV)
    f.gemm_nt_bf16_fused(a, b, bias=bias, activation=name, preact=pre)
    ga, gb, gbias = f.gemm_nt_bf16_fused_backward(G, a, b, activation=name, preact=None if name == "none" else pre,
                                                  bias_grad=True)
    z, _, tight, hw = F.fused_reference(a, b, bias=bias)
    g64 = G.cpu().double()
    dz = g64 * F.act(name, z)[1]
    err = grad_error(name, g64, z, tight + hw)
    F.check(ga, *F.backward_products(dz, err, b), N, f"grad_a {name}")
    F.check(gb, *F.backward_products(dz.t(), err.t(), a), M, f"grad_b {name}")
    # FP32 sums of M terms in an order of depth at most M / 64 + 32: a thread's rows of a block (up to 8), 8 threads, every
    # 8th block (of 8 rows or more each), 8 threads
    tol = err.sum(0) + (M / 64 + 32) * 2.0 ** -24 * dz.abs().sum(0) + 2.0 ** -23 * dz.abs().sum(0)
    assert ((gbias.cpu().double() - dz.sum(0)).abs() <= tol).all()


@pytest.mark.parametrize("M,N,K", BF_SHAPES)
@pytest.mark.parametrize("name", F.ACTS)
def test_gated_bf16_backward(f, M, N, K, name):
    a, G = rand(M + K, M, K), rand(9, M, N)
    wg, wu = rand(N + 7 * K, N, K, std=0.25), rand(N + 5 * K, N, K, std=0.25)
    pre = torch.empty((2, M, N), device=DEV)
    f.gated_nt_bf16(a, wg, wu, activation=name, preact=pre)
    ga, gg, gu = f.gated_nt_bf16_backward(G, a, wg, wu, pre, activation=name)
    (g, Sg, hg), (u, Su, hu) = F.product(a, wg), F.product(a, wu)
    eg, eu = 1e-5 * Sg + hg, 1e-5 * Su + hu
    g64 = G.cpu().double()
    v, dv = F.act(name, g)
    dp, du = g64 * u * dv, g64 * v
    err_p = grad_error(name, g64 * u, g, eg) + 1.2 * (g64.abs() * eu)
    err_u = g64.abs() * (1.2 * eg + 2.0 ** -19 * g.abs())
    p, q = F.backward_products(dp, err_p, wg), F.backward_products(du, err_u, wu)
    F.check(ga, *(x + y for x, y in zip(p, q)), N, f"grad_a {name}")
    F.check(gg, *F.backward_products(dp.t(), err_p.t(), a), M, f"grad_gate {name}")
    F.check(gu, *F.backward_products(du.t(), err_u.t(), a), M, f"grad_up {name}")


# Every class of the kernels with ragged edges, by the plan (variant; the few-token kernel's weight rows and 16-token
# blocks): (op, M, N, K), with a short K so that the 64-bit reference stays small.
CLASS_CASES = [
    (0, 4000, 2050, 272, 1, 0, 0), (0, 130, 17001, 272, 2, 0, 0), (0, 2050, 77, 272, 7, 0, 0), (0, 1, 77, 272, 4, 16, 1),
    (0, 20, 77, 272, 4, 16, 2), (0, 40, 77, 272, 4, 16, 4), (0, 1, 5003, 272, 4, 32, 1), (0, 20, 9003, 272, 4, 32, 2),
    (0, 130, 2503, 272, 4, 32, 4), (0, 1, 17003, 272, 4, 64, 1), (0, 32, 14339, 4096, 4, 64, 2), (0, 40, 9001, 272, 4, 64, 4),
    (1, 130, 17001, 272, 1, 0, 0), (1, 130, 9001, 272, 2, 0, 0), (1, 2050, 77, 272, 7, 0, 0), (1, 1, 77, 272, 4, 16, 1),
    (1, 20, 77, 272, 4, 16, 2), (1, 40, 77, 272, 4, 16, 4), (1, 1, 9003, 272, 4, 32, 1), (1, 40, 4101, 272, 4, 32, 4),
    (2, 4000, 2050, 200, 1, 0, 0), (2, 130, 17001, 200, 2, 0, 0), (2, 2050, 77, 200, 7, 0, 0), (2, 1, 77, 200, 4, 16, 1),
    (2, 20, 77, 200, 4, 16, 2), (2, 40, 77, 200, 4, 16, 4), (2, 1, 5003, 200, 4, 32, 1), (2, 20, 9003, 200, 4, 32, 2),
    (2, 130, 2503, 200, 4, 32, 4), (2, 1, 17003, 200, 4, 64, 1), (2, 40, 9001, 200, 4, 64, 4),
    (3, 130, 17001, 200, 1, 0, 0), (3, 130, 9001, 200, 2, 0, 0), (3, 2050, 77, 200, 7, 0, 0), (3, 1, 77, 200, 4, 16, 1),
    (3, 20, 77, 200, 4, 16, 2), (3, 40, 77, 200, 4, 16, 4), (3, 1, 9003, 200, 4, 32, 1), (3, 40, 4101, 200, 4, 32, 4)]


@pytest.mark.parametrize("op,M,N,K,variant,rows,blocks", CLASS_CASES)
def test_every_class(f, op, M, N, K, variant, rows, blocks):
    p = f.fused_plan(op, M, N, K)
    assert p.variant == variant and (variant != 4 or (p.tile_n, p.token_blocks) == (rows, blocks))
    dt = E4 if op < 2 else BF
    a, b = rand(1, M, K, dtype=dt), rand(2, N, K, dtype=dt, std=0.25)
    if op in (0, 2):
        bias, res = rand(3, N, dtype=torch.float32), rand(4, M, N)
        call = f.gemm_nt_fused if op == 0 else f.gemm_nt_bf16_fused
        out = call(a, b, bias=bias, activation="gelu", residual=res)
        _, v, tight, hw = F.fused_reference(a, b, bias=bias, name="gelu", res=res)
    else:
        u = rand(5, N, K, dtype=dt, std=0.25)
        out = (f.gated_nt if op == 1 else f.gated_nt_bf16)(a, b, u, activation="silu")
        _, _, v, tight, hw = F.gated_reference(a, b, u)
    F.check(out, v, tight, hw, K, f"op {op}")


@pytest.mark.parametrize("M,N,K,va,vb", [(4000, 72, 3000, 1, 7), (2000, 205, 2056, 2, 7), (72, 4000, 3000, 7, 1),
                                         (200, 2000, 2056, 7, 2), (300, 400, 520, 7, 7)])
def test_every_backward_class(f, M, N, K, va, vb):
    """grad_a is M x K reduced over N, grad_b N x K reduced over M."""
    cols = (N + 63) // 64 * 64
    assert f.fused_plan(4, M, K, cols).variant == va and f.fused_plan(4, N, K, M).variant == vb
    a, b, G = rand(1, M, K), rand(2, N, K, std=0.25), rand(3, M, N)
    z = rand(4, M, N, dtype=torch.float32)
    ga, gb, _ = f.gemm_nt_bf16_fused_backward(G, a, b, activation="silu", preact=z)
    g64, z64 = G.cpu().double(), z.cpu().double()
    dz = g64 * F.act("silu", z64)[1]
    err = grad_error("silu", g64, z64, torch.zeros_like(z64))
    F.check(ga, *F.backward_products(dz, err, b), N, "grad_a")
    F.check(gb, *F.backward_products(dz.t(), err.t(), a), M, "grad_b")


@pytest.mark.parametrize("M,N,K,va,vw", [(4000, 36, 3000, 1, 7), (72, 2000, 3000, 7, 1)])
def test_every_gated_backward_class(f, M, N, K, va, vw):
    cols = (N + 63) // 64 * 64
    assert f.fused_plan(4, M, K, 2 * cols).variant == va and f.fused_plan(4, 2 * N, K, M).variant == vw
    a, wg, wu, G = rand(1, M, K), rand(2, N, K, std=0.25), rand(5, N, K, std=0.25), rand(3, M, N)
    pre = rand(4, 2 * M, N, dtype=torch.float32).view(2, M, N)
    ga, gg, gu = f.gated_nt_bf16_backward(G, a, wg, wu, pre)
    g64, (g, u) = G.cpu().double(), pre.cpu().double()
    v, dv = F.act("silu", g)
    dp, du = g64 * u * dv, g64 * v
    ep, eu = grad_error("silu", g64 * u, g, torch.zeros_like(g)), g64.abs() * 2.0 ** -19 * g.abs()
    F.check(ga, *(x + y for x, y in zip(F.backward_products(dp, ep, wg), F.backward_products(du, eu, wu))), N, "grad_a")
    F.check(gg, *F.backward_products(dp.t(), ep.t(), a), M, "grad_gate")
    F.check(gu, *F.backward_products(du.t(), eu.t(), a), M, "grad_up")


@pytest.mark.parametrize("M,N,K", [(5, 9000, 264), (130, 4100, 136), (6000, 40, 136), (9000, 130, 520), (12000, 1030, 1032)])
def test_split_backward_products(f, M, N, K):
    """Few output tiles and a long sum: K split over workgroups, for grad_a (reduced over N) or the weights' (over M)."""
    cols = (N + 63) // 64 * 64
    splits = f.fused_plan(4, M, K, cols).k_splits, f.fused_plan(4, N, K, M).k_splits
    assert max(splits) > 1
    a, b, u, G = rand(1, M, K), rand(2, N, K, std=0.25), rand(5, N, K, std=0.25), rand(3, M, N)
    pre = rand(4, 2 * M, N, dtype=torch.float32).view(2, M, N)
    g64, (z, w) = G.cpu().double(), pre.cpu().double()
    v, dv = F.act("silu", z)
    zero = torch.zeros_like(z)
    ga, gb, _ = f.gemm_nt_bf16_fused_backward(G, a, b, "silu", pre[0])
    dz, err = g64 * dv, grad_error("silu", g64, z, zero)
    F.check(ga, *F.backward_products(dz, err, b), N, "grad_a")
    F.check(gb, *F.backward_products(dz.t(), err.t(), a), M, "grad_b")
    for _ in range(3):
        again = f.gemm_nt_bf16_fused_backward(G, a, b, "silu", pre[0])
        assert torch.equal(again[0], ga) and torch.equal(again[1], gb)
    ga, gg, gu = f.gated_nt_bf16_backward(G, a, b, u, pre)
    dp, du = g64 * w * dv, g64 * v
    ep, eu = grad_error("silu", g64 * w, z, zero), g64.abs() * 2.0 ** -19 * z.abs()
    F.check(ga, *(x + y for x, y in zip(F.backward_products(dp, ep, b), F.backward_products(du, eu, u))), N, "grad_a")
    F.check(gg, *F.backward_products(dp.t(), ep.t(), a), M, "grad_gate")
    F.check(gu, *F.backward_products(du.t(), eu.t(), a), M, "grad_up")
