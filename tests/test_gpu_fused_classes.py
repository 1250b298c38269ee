"""Every build of the fused and gated kernels, forced by its size and asserted
by the plan, on sums long enough that every ring slot is refilled, with K a
multiple of a K step and not: all operand types, scale layouts, activations and
residual layouts.  Selected rows and columns, the tiles' edges among them, are
compared with 64-bit references (tests/_fused.py)."""
import pytest
import torch

from tests import _fused as F
from tests.test_gpu_fused import BF, DEV, E4, E5, f, grad_error, rand, scales, strided  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu


def pick(n, seed, most=320):
    """Indexes of up to `most` rows or columns: both ends, the neighbourhoods of the tiles' edges, and random ones."""
    if n <= most:
        return torch.arange(n, device=DEV)
    keep = set(range(40)) | set(range(n - 60, n)) | {e + d for e in range(64, n, max(64, n // 8 // 64 * 64)) for d in (-1, 0)}
    g = torch.Generator().manual_seed(seed)
    for i in torch.randperm(n, generator=g).tolist():
        if len(keep) >= most:
            break
        keep.add(i)
    return torch.tensor(sorted(keep), device=DEV)


def some(t, idx):
    return t if t is None or t.numel() == 1 else t[idx]


# (tokens, weights, activation, row scales, channel scales, bias, residual)
FP8 = [(E4, E4, "none", "each", "each", True, "whole"), (E4, E5, "relu", "one", "each", False, "unaligned"),
       (E5, E4, "silu", None, "one", True, "in place"), (E5, E5, "gelu", "each", None, False, None),
       (E4, E4, "gelu_tanh", "each", "each", True, "in place")]


def scale(kind, seed, n):
    return None if kind is None else scales(seed, n if kind == "each" else 1)


def residual_and_out(kind, M, N):
    """(residual, the same values kept, out)."""
    if kind is None:
        return None, None, None
    res = rand(4, M, N)
    if kind == "in place":
        out = torch.full((M, (N + 7) // 8 * 8 + 8), 7.0, dtype=BF, device=DEV)
        out[:, :N] = res
        return out[:, :N], res, out[:, :N]
    return (strided(res, 3) if kind == "unaligned" else strided(res, 8 - N % 8)), res, None


def check_plan(f, op, M, N, K, want):
    p = f.fused_plan(op, M, N, K)
    assert ((p.variant, p.tile_n, p.token_blocks) if p.variant == 4 else p.variant) == want


def check_fused(f, op, M, N, K, case):
    ta, tb, name, ka, kb, with_bias, kind = case
    a, b = rand(1, M, K, dtype=ta), rand(2, N, K, dtype=tb, std=0.25)
    sa, sb = scale(ka, 5, M), scale(kb, 6, N)
    bias = rand(3, N, dtype=torch.float32) if with_bias else None
    res, kept, out = residual_and_out(kind, M, N)
    if op == 0:
        got = f.gemm_nt_fused(a, b, sa, sb, bias=bias, activation=name, residual=res, out=out)
        pre = None
    else:
        pre = torch.full((M, N + (3 if kind == "unaligned" else -N % 4)), 9.0, device=DEV)
        got = f.gemm_nt_bf16_fused(a, b, bias=bias, activation=name, residual=res, out=out, preact=pre[:, :N])
        assert (pre[:, N:] == 9).all()
    if out is not None:
        assert (out._base[:, N:] == 7).all()
    r, c = pick(M, 1), pick(N, 2)
    z, v, tight, hw = F.fused_reference(a.view(torch.uint8)[r].view(ta) if op == 0 else a[r],
                                        b.view(torch.uint8)[c].view(tb) if op == 0 else b[c],
                                        some(sa, r), some(sb, c), some(bias, c), name,
                                        None if kept is None else kept[r][:, c])
    F.check(got[r][:, c], v, tight, hw, K, f"{case}")
    if pre is not None:
        assert ((pre[r][:, c].cpu().double() - z).abs() <= tight + hw).all()


def check_gated(f, op, M, N, K, case):
    ta, tb, name, ka, kb, _, kind = case
    a, g, u = rand(1, M, K, dtype=ta), rand(2, N, K, dtype=tb, std=0.25), rand(3, N, K, dtype=tb, std=0.25)
    sa, sg, su = scale(ka, 5, M), scale(kb, 6, N), scale(kb, 7, N)
    r, c = pick(M, 1), pick(N, 2)
    if op == 1:
        got = f.gated_nt(a, g, u, sa, sg, su, activation=name)
        a, g, u = (t.view(torch.uint8)[i].view(t.dtype) for t, i in ((a, r), (g, c), (u, c)))
    else:
        pre = torch.full((2, M, N + (3 if kind == "unaligned" else -N % 4)), 9.0, device=DEV)
        got = f.gated_nt_bf16(a, g, u, activation=name, preact=pre[:, :, :N])
        assert (pre[:, :, N:] == 9).all()
        a, g, u = a[r], g[c], u[c]
        for p, w in zip(pre, (g, u)):
            z, S, h = F.product(a, w)
            assert ((p[r][:, c].cpu().double() - z).abs() <= 1e-5 * S + h).all()
    _, _, v, tight, hw = F.gated_reference(a, g, u, some(sa, r), some(sg, c), some(su, c), name)
    F.check(got[r][:, c], v, tight, hw, K, f"{case}")


def cases(op):
    return FP8 if op < 2 else [(BF, BF, name, None, None, b, kind) for _, _, name, _, _, b, kind in FP8]


# 16 and 17 K steps of 128 bytes: at least 4 for each of the few-token kernel's waves, whose rings have 2 or 3 slots
FEW = [(0, 1, 77, (4, 16, 1)), (0, 32, 77, (4, 16, 2)), (0, 37, 77, (4, 16, 4)), (0, 16, 9001, (4, 32, 1)),
       (0, 32, 9001, (4, 32, 2)), (0, 130, 2503, (4, 32, 4)), (0, 1, 17003, (4, 64, 1)), (0, 32, 14339, (4, 64, 2)),
       (0, 48, 9001, (4, 64, 4)), (0, 600, 333, (4, 16, 4)),
       (1, 1, 77, (4, 16, 1)), (1, 32, 77, (4, 16, 2)), (1, 37, 77, (4, 16, 4)), (1, 16, 9001, (4, 32, 1)),
       (1, 32, 14339, (4, 32, 2)), (1, 48, 4101, (4, 32, 4)), (1, 600, 333, (4, 16, 4))]
FEW += [(op + 2, M, N, want) for op, M, N, want in FEW]


@pytest.mark.parametrize("op,M,N,want", FEW)
def test_few_tokens(f, op, M, N, want):
    for K in ((2048, 2064) if op < 2 else (1024, 1032)):
        check_plan(f, op, M, N, K, want)
        for case in cases(op):
            (check_gated if op % 2 else check_fused)(f, op, M, N, K, case)


# 8 and 9 K steps: more than the 2 to 4 slots of the tiles' rings
TILES = [(0, 2100, 1003, 7), (0, 4000, 4100, 2), (0, 2100, 4100, 1), (1, 2100, 500, 7), (1, 4000, 2050, 2), (1, 2100, 2050, 1),
         (2, 2100, 1003, 7), (2, 4000, 4100, 2), (2, 2100, 4100, 1), (3, 2100, 500, 7), (3, 4000, 2050, 2), (3, 2100, 2050, 1)]


@pytest.mark.parametrize("op,M,N,want", TILES)
@pytest.mark.parametrize("whole_steps", [True, False])
def test_tiles(f, op, M, N, want, whole_steps):
    K = (1024 if whole_steps else 1040) // (1 if op < 2 else 2)
    check_plan(f, op, M, N, K, want)
    for case in cases(op):
        (check_gated if op % 2 else check_fused)(f, op, M, N, K, case)


@pytest.mark.parametrize("op,M,N,want", [t for t in TILES if t[0] in (0, 2)])
def test_tiles_of_empty_sums(f, op, M, N, want):
    """K = 0 on sizes past the few-token kernel's: act(bias) + residual."""
    M = max(M, 2100)
    a, b = (torch.zeros(n, 0, dtype=E4 if op == 0 else BF, device=DEV) for n in (M, N))
    bias, res = rand(3, N, dtype=torch.float32), rand(4, M, N)
    assert f.fused_plan(op, M, N, 0).variant in (1, 2, 7)
    got = (f.gemm_nt_fused if op == 0 else f.gemm_nt_bf16_fused)(a, b, bias=bias, activation="silu", residual=res)
    z, r = bias.cpu().double(), res.cpu().double()
    v = F.act("silu", z)[0]
    assert ((got.cpu().double() - v - r).abs() <= F.EPS * (v + r).abs() + 2.0 ** -19 * z.abs() + 2.0 ** -24 * r.abs()).all()


# The gated form's backward pass: the class of its token gradient (over both matrices' columns) and of its weight
# gradients (two products in one launch), and whether their sums are split.
PAIRS = [(72, 36, 136, 7, 7, (False, False)), (1030, 36, 136, 7, 7, (False, True)),
         (4000, 36, 1032, 2, 7, (False, True)), (4000, 36, 2056, 1, 7, (False, True)),
         (9000, 36, 2056, 2, 2, (False, True)), (9000, 130, 2056, 2, 1, (False, True)),
         (72, 520, 136, 7, 7, (True, False)), (72, 2000, 1032, 7, 2, (True, False)),
         (72, 2000, 2056, 7, 1, (True, False)), (520, 4000, 2056, 2, 2, (True, False)),
         (9000, 4000, 136, 1, 2, (True, True))]


@pytest.mark.parametrize("M,N,K,va,vw,split", PAIRS)
def test_gated_backward_classes(f, M, N, K, va, vw, split):
    cols = (N + 63) // 64 * 64
    pa, pw = f.fused_plan(4, M, K, 2 * cols), f.fused_plan(4 + f.PLAN_PAIR, N, K, M)
    assert (pa.variant, pw.variant) == (va, vw) and (pa.k_splits > 1, pw.k_splits > 1) == split
    a, wg, wu, G = rand(1, M, K), rand(2, N, K, std=0.25), rand(5, N, K, std=0.25), rand(3, M, N)
    pre = rand(4, 2 * M, N, dtype=torch.float32).view(2, M, N)
    ga, gg, gu = f.gated_nt_bf16_backward(G, a, wg, wu, pre)
    g64, (g, u) = G.cpu().double(), pre.cpu().double()
    v, dv = F.act("silu", g)
    dp, du = g64 * u * dv, g64 * v
    ep, eu = grad_error("silu", g64 * u, g, torch.zeros_like(g)), g64.abs() * 2.0 ** -19 * g.abs()
    r, n, k = pick(M, 1).cpu(), pick(N, 2).cpu(), pick(K, 3).cpu()
    F.check(ga.cpu()[r], *(x + y for x, y in zip(F.backward_products(dp[r], ep[r], wg), F.backward_products(du[r], eu[r], wu))),
            N, "grad_a")
    F.check(gg.cpu()[n][:, k], *F.backward_products(dp.t()[n], ep.t()[n], a[:, k.to(DEV)]), M, "grad_gate")
    F.check(gu.cpu()[n][:, k], *F.backward_products(du.t()[n], eu.t()[n], a[:, k.to(DEV)]), M, "grad_up")


@pytest.mark.parametrize("M,N,K", [(2100, 1000, 520), (300, 4104, 136)])
def test_output_gradient_as_operand(f, M, N, K):
    """Without an activation the output's gradient itself is the operand, also where its rows end inside a K step."""
    a, b, G = rand(1, M, K), rand(2, N, K, std=0.25), rand(3, M, N)
    ga, gb, _ = f.gemm_nt_bf16_fused_backward(strided(G, 8), a, b)
    g64 = G.cpu().double()
    zero = torch.zeros_like(g64)
    F.check(ga, *F.backward_products(g64, zero, b), N, "grad_a")
    F.check(gb, *F.backward_products(g64.t(), zero.t(), a), M, "grad_b")
