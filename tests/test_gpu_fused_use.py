"""The fused and gated products as they are used: strided operands, in-place
residuals, streams and graphs, empty sizes, extreme values, long offsets, and a
feed-forward block run forward and backward.  References: tests/_fused.py."""
import math

import pytest
import torch

from tests import _fused as F
from tests.test_gpu_fused import BF, DEV, E4, E5, f, rand, scales, strided  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu


def wide(t, extra):
    """The same values in rows `extra` elements longer, whose ends hold NaN (the row stride stays a multiple of 16 bytes)."""
    return strided(t, extra)


@pytest.mark.parametrize("M,N,K", [(5, 37, 208), (40, 130, 272), (300, 261, 144), (1500, 1030, 80)])
def test_strided_fp8(f, M, N, K):
    a, b, u = (rand(s, r, K, dtype=E4, std=0.5) for s, r in ((1, M), (2, N), (3, N)))
    sa, sb = scales(4, M), scales(5, N)
    res = rand(6, M, N)
    want = f.gemm_nt_fused(a, b, sa, sb, activation="silu", residual=res)
    gated = f.gated_nt(a, b, u, sa, sb, sb)
    wa, wb, wu = wide(a, 16), wide(b, 48), wide(u, 32)
    for r in (res, wide(res, 3), wide(res, 8)):
        out = torch.full((M, N + 24 - N % 8), 7.0, dtype=BF, device=DEV)
        f.gemm_nt_fused(wa, wb, sa, sb, activation="silu", residual=r, out=out[:, :N])
        assert torch.equal(out[:, :N], want) and (out[:, N:] == 7).all()
    out = torch.full((M, N + 24 - N % 8), 7.0, dtype=BF, device=DEV)
    f.gated_nt(wa, wb, wu, sa, sb, sb, out=out[:, :N])
    assert torch.equal(out[:, :N], gated) and (out[:, N:] == 7).all()
    # the halves of a merged weight
    both = torch.cat((b.view(torch.uint8), u.view(torch.uint8))).view(E4)
    assert torch.equal(f.gated_nt(a, both[:N], both[N:], sa, sb, sb), gated)


@pytest.mark.parametrize("M,N,K", [(5, 37, 104), (40, 130, 136), (300, 261, 72), (1500, 1030, 40)])
def test_strided_bf16(f, M, N, K):
    a, b, u = (rand(s, r, K, std=0.5) for s, r in ((1, M), (2, N), (3, N)))
    G = rand(7, M, N)
    pre, pre2 = torch.empty(M, N, device=DEV), torch.empty(2, M, N, device=DEV)
    want = f.gemm_nt_bf16_fused(a, b, activation="gelu", preact=pre)
    ga, gb, gbias = f.gemm_nt_bf16_fused_backward(G, a, b, activation="gelu", preact=pre, bias_grad=True)
    h = f.gated_nt_bf16(a, b, u, preact=pre2)
    gated = f.gated_nt_bf16_backward(G, a, b, u, pre2)
    wa, wb, wu = wide(a, 8), wide(b, 24), wide(u, 24)
    for extra in (1, 3, 4):
        wp = torch.full((M, N + extra), math.nan, device=DEV)
        out = f.gemm_nt_bf16_fused(wa, wb, activation="gelu", preact=wp[:, :N])
        assert torch.equal(out, want) and torch.equal(wp[:, :N], pre) and wp[:, N:].isnan().all()
        got = f.gemm_nt_bf16_fused_backward(wide(G, extra), wa, wb, activation="gelu", preact=wp[:, :N], bias_grad=True)
        for x, y in zip(got, (ga, gb, gbias)):
            assert torch.equal(x, y)
        wp2 = torch.full((2, M + 1, N + extra), math.nan, device=DEV)[:, :M, :N]
        assert torch.equal(f.gated_nt_bf16(wa, wb, wu, preact=wp2), h) and torch.equal(wp2, pre2)
        for x, y in zip(f.gated_nt_bf16_backward(wide(G, extra), wa, wb, wu, wp2), gated):
            assert torch.equal(x, y)


@pytest.mark.parametrize("M", [1, 37, 64, 200, 1000])
@pytest.mark.parametrize("N", [256, 333])
def test_residual_in_place(f, M, N):
    K = 144
    a, b = rand(1, M, K, dtype=E4), rand(2, N, K, dtype=E4)
    x, y = rand(3, M, K), rand(4, N, K)
    stream = torch.zeros((M, (N + 7) // 8 * 8), dtype=BF, device=DEV)[:, :N]
    stream.copy_(rand(5, M, N))
    before = stream.clone()
    want = f.gemm_nt_fused(a, b, residual=before)
    assert f.gemm_nt_fused(a, b, residual=stream, out=stream) is stream and torch.equal(stream, want)
    want = f.gemm_nt_bf16_fused(x, y, activation="relu", residual=want)
    f.gemm_nt_bf16_fused(x, y, activation="relu", residual=stream, out=stream)
    assert torch.equal(stream, want)


def test_gradients_on_request(f):
    M, N, K = 70, 90, 88
    a, b, u, G = rand(1, M, K), rand(2, N, K), rand(3, N, K), rand(4, M, N)
    pre = torch.empty(M, N, device=DEV)
    f.gemm_nt_bf16_fused(a, b, activation="silu", preact=pre)
    full = f.gemm_nt_bf16_fused_backward(G, a, b, "silu", pre, bias_grad=True)
    for want in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        got = f.gemm_nt_bf16_fused_backward(G, a, b, "silu", pre, a_grad=want[0], b_grad=want[1], bias_grad=want[2])
        for w, x, y in zip(want, got, full):
            assert (x is None) if not w else torch.equal(x, y)
    # no activation: the output's gradient itself, also through the workspace (odd columns, unaligned rows)
    for n in (88, 90):
        ga, gb, gbias = f.gemm_nt_bf16_fused_backward(G[:, :n], a, b[:n], bias_grad=True)
        g64 = G[:, :n].cpu().double()
        F.check(ga, *F.backward_products(g64, torch.zeros_like(g64), b[:n]), n, "grad_a")
        F.check(gb, *F.backward_products(g64.t(), torch.zeros_like(g64).t(), a), M, "grad_b")
        assert ((gbias.cpu().double() - g64.sum(0)).abs() <= 34 * 2.0 ** -24 * g64.abs().sum(0)).all()   # depth M / 64 + 32
    pre2 = torch.empty(2, M, N, device=DEV)
    f.gated_nt_bf16(a, b, u, preact=pre2)
    full = f.gated_nt_bf16_backward(G, a, b, u, pre2)
    ga, gg, gu = f.gated_nt_bf16_backward(G, a, b, u, pre2, w_grad=False)
    assert torch.equal(ga, full[0]) and gg is None and gu is None
    ga, gg, gu = f.gated_nt_bf16_backward(G, a, b, u, pre2, a_grad=False)
    assert ga is None and torch.equal(gg, full[1]) and torch.equal(gu, full[2])


def test_empty_sizes(f):
    z8 = lambda *s: torch.zeros(*s, device=DEV).to(E4)  # noqa: E731
    zb = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
    assert f.gemm_nt_fused(z8(0, 32), z8(5, 32)).shape == (0, 5) and f.gated_nt(z8(3, 32), z8(0, 32), z8(0, 32)).shape == (3, 0)
    bias, res = rand(1, 40, dtype=torch.float32), rand(2, 100, 40)
    for M in (3, 100):
        # K = 0: the empty sum
        want = (torch.nn.functional.silu(bias) + res[:M].float()).bfloat16()
        got = f.gemm_nt_fused(z8(M, 0), z8(40, 0), bias=bias, activation="silu", residual=res[:M])
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
        pre = torch.full((M, 40), 9.0, device=DEV)
        got = f.gemm_nt_bf16_fused(zb(M, 0), zb(40, 0), bias=bias, activation="silu", residual=res[:M], preact=pre)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
        assert torch.equal(pre, bias.expand(M, 40))
        assert (f.gated_nt(z8(M, 0), z8(40, 0), z8(40, 0)) == 0).all()
        assert (f.gated_nt_bf16(zb(M, 0), zb(40, 0), zb(40, 0)) == 0).all()
        ga, gb, gbias = f.gemm_nt_bf16_fused_backward(res[:M], zb(M, 0), zb(40, 0), "silu", pre, bias_grad=True)
        assert ga.shape == (M, 0) and gb.shape == (40, 0)
        dz = res[:M].cpu().double() * F.act("silu", pre.cpu().double())[1]
        assert ((gbias.cpu().double() - dz.sum(0)).abs() <= 1e-5 * dz.abs().sum(0)).all()
    # no rows: zero weight and bias gradients; no columns: a zero token gradient
    ga, gb, gbias = f.gemm_nt_bf16_fused_backward(zb(0, 24), zb(0, 32), rand(3, 24, 32), bias_grad=True)
    assert ga.shape == (0, 32) and (gb == 0).all() and (gbias == 0).all()
    ga, gg, gu = f.gated_nt_bf16_backward(zb(0, 24), zb(0, 32), rand(3, 24, 32), rand(4, 24, 32), torch.empty(2, 0, 24, device=DEV))
    assert (gg == 0).all() and (gu == 0).all()
    ga, gb, _ = f.gemm_nt_bf16_fused_backward(zb(9, 0), rand(3, 9, 32), zb(0, 32))
    assert (ga == 0).all() and gb.shape == (0, 32)
    ga, _, _ = f.gated_nt_bf16_backward(zb(9, 0), rand(3, 9, 32), zb(0, 32), zb(0, 32), torch.empty(2, 9, 0, device=DEV))
    assert (ga == 0).all()


@pytest.mark.parametrize("M", [3, 100, 1200])
def test_extreme_values(f, M):
    """Saturated activations stay finite and exact at both ends; NaN and infinity stay in their row or column."""
    K, N = 16, 300
    zs = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, -3.0, -9.0, 9.0, -40.0, 40.0, -1e4, 1e4, -3e38, 3e38, -88.0, -104.0])
    bias = zs.repeat(N)[:N].to(DEV)
    x, w = torch.zeros(M, K, dtype=BF, device=DEV), torch.zeros(N, K, dtype=BF, device=DEV)
    G = torch.ones(M, N, dtype=BF, device=DEV)
    for name in F.ACTS:
        pre = torch.empty(M, N, device=DEV)
        out = f.gemm_nt_bf16_fused(x, w, bias=bias, activation=name, preact=pre)
        v, dv = F.act(name, bias.cpu().double().clamp(-1e10, 1e10))
        v = torch.where(bias.cpu().double() > 1e10, bias.cpu().double(), v)
        if name == "none":
            v = bias.cpu().double()
        assert (pre == bias).all() and not out.isnan().any(), name
        # One rounding, 2^-18 relative for exp of arguments up to 100 (2^-24 of them).  The sigmoid is the reciprocal of
        # 1 + exp(-v), and a reciprocal below FP32's normal range, 2^-126, is returned as 0: so z times it is off by up
        # to 2^-126 |z|.  That happens only while exp(-v) is finite, -v < 89; for the tanh form of GELU v <= z below 0,
        # so |z| < 89 there too (and past it both sides are 0).  The inputs' -88 gives 88 2^-126 = 1.04e-36.
        tol = F.EPS * v.abs() + 2.0 ** -16 * v.abs() + 2.0 ** -126 * bias.cpu().double().abs().clamp(max=89)
        assert ((out.cpu().double() - v).abs() <= tol).all(), name
        _, _, gbias = f.gemm_nt_bf16_fused_backward(G, x, w, name, None if name == "none" else pre, bias_grad=True)
        assert ((gbias.cpu().double() - M * dv).abs() <= M * (1e-6 + 4e-5 * dv.abs())).all(), name
    x, w = rand(1, M, 64), rand(2, N, 64)
    want = f.gemm_nt_bf16_fused(x, w, activation="silu")
    x[1, 5], w[7, 3] = math.nan, math.inf
    got = f.gemm_nt_bf16_fused(x, w, activation="silu")
    keep = torch.ones(M, N, dtype=torch.bool, device=DEV)
    keep[1], keep[:, 7] = False, False
    assert torch.equal(got[keep], want[keep]) and got[1].isnan().all() and not torch.isfinite(got[:, 7]).all()
    u = rand(3, N, 64)
    ok = f.gated_nt_bf16(rand(1, M, 64), rand(2, N, 64), u)
    got = f.gated_nt_bf16(x, w, u)
    assert torch.equal(got[keep], ok[keep]) and got[1].isnan().all()


def block(f, x, wg, wu, wd, dy):
    """A feed-forward block with residual, forward and backward: (y, grad_x, grad_wg, grad_wu, grad_wd)."""
    pre = torch.empty(2, x.shape[0], wg.shape[0], device=x.device)
    h = f.gated_nt_bf16(x, wg, wu, preact=pre)
    y = f.gemm_nt_bf16_fused(h, wd, residual=x)
    dh, dwd, _ = f.gemm_nt_bf16_fused_backward(dy, h, wd)
    dx, dwg, dwu = f.gated_nt_bf16_backward(dh, x, wg, wu, pre)
    return y, dx, dwg, dwu, dwd


def block_operands(T, D, H, seed=0):
    return (rand(seed + 1, T, D), rand(seed + 2, H, D, std=D ** -0.5), rand(seed + 3, H, D, std=D ** -0.5),
            rand(seed + 4, D, H, std=H ** -0.5), rand(seed + 5, T, D))


@pytest.mark.parametrize("T,D,H", [(1, 64, 160), (50, 136, 344), (333, 256, 680), (1024, 512, 1368)])
def test_feed_forward_block(f, T, D, H):
    x, wg, wu, wd, dy = block_operands(T, D, H)
    got = block(f, x, wg, wu, wd, dy)
    x6, g6, u6, d6, dy6 = (t.cpu().double() for t in (x, wg, wu, wd, dy))
    g, u = x6 @ g6.t(), x6 @ u6.t()
    v, dv = F.act("silu", g)
    h = v * u
    dh = dy6 @ d6
    dg, du = dh * u * dv, dh * v
    want = (h @ d6.t() + x6, dg @ g6 + du @ u6, dg.t() @ x6, du.t() @ x6, dy6.t() @ h)
    # y: h rounded and y rounded, dx and dw: dh, dg or du, and the result: at most four roundings of eps in a row
    for a, b, name in zip(got, want, ("y", "dx", "dwg", "dwu", "dwd")):
        rel = float((a.cpu().double() - b).norm() / b.norm())
        assert rel <= 4 * F.EPS, (name, rel)


def test_gradients_against_differences(f):
    """<grad, direction> against central differences of sum(G * out) in 64 bits, for each input."""
    M, N, K, h = 60, 72, 80, 1e-5
    a, b, u, G = rand(1, M, K), rand(2, N, K, std=0.1), rand(3, N, K, std=0.1), rand(4, M, N)
    bias = rand(5, N, dtype=torch.float32)
    a6, b6, u6, G6, c6 = (t.cpu().double() for t in (a, b, u, G, bias))
    for name in ("silu", "gelu", "gelu_tanh"):
        pre, pre2 = torch.empty(M, N, device=DEV), torch.empty(2, M, N, device=DEV)
        f.gemm_nt_bf16_fused(a, b, bias=bias, activation=name, preact=pre)
        f.gated_nt_bf16(a, b, u, activation=name, preact=pre2)
        fused = f.gemm_nt_bf16_fused_backward(G, a, b, name, pre, bias_grad=True)
        gated = f.gated_nt_bf16_backward(G, a, b, u, pre2, name)
        loss = lambda x, w, c: (G6 * F.act(name, x @ w.t() + c)[0]).sum()  # noqa: E731
        loss2 = lambda x, w, v: (G6 * F.act(name, x @ w.t())[0] * (x @ v.t())).sum()  # noqa: E731
        for fn, at, grads in ((loss, (a6, b6, c6), fused), (loss2, (a6, b6, u6), gated)):
            for i, grad in enumerate(grads):
                g = grad.cpu().double()
                d = torch.randn(at[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
                up = fn(*(t + h * d if k == i else t for k, t in enumerate(at)))
                down = fn(*(t - h * d if k == i else t for k, t in enumerate(at)))
                # each entry off by at most two roundings of its terms, in directions that do not depend on d: a
                # random sum of them, six standard deviations wide
                tol = 6 * 2 * F.EPS * float((g * d).norm()) + 1e-4 * abs(float(up - down)) / (2 * h)
                assert abs(float((g * d).sum()) - float(up - down) / (2 * h)) <= tol, (name, i)


def test_streams(f):
    """Two streams at once, each with its own operands, against the same calls one after the other."""
    sets = [block_operands(300, 256, 688, seed=10 * s) for s in range(2)]
    want = [block(f, *s) for s in sets]
    q8 = [(rand(1 + s, 33, 256, dtype=E4), rand(3 + s, 512, 256, dtype=E4)) for s in range(2)]
    want8 = [f.gemm_nt_fused(*q, activation="gelu") for q in q8]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got, got8 = [[], []], [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(block(f, *sets[i]))
                got8[i].append(f.gemm_nt_fused(*q8[i], activation="gelu"))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for r in got[i] for x, y in zip(r, want[i]))
        assert all(torch.equal(x, want8[i]) for x in got8[i])


def test_graphs(f):
    """Two captured training steps and a captured decode call, replayed in turn with eager calls between, on new inputs."""
    operands = block_operands(130, 256, 344)
    x8, w8 = rand(7, 5, 256, dtype=E4), rand(8, 96, 256, dtype=E4)
    block(f, *operands)
    f.gemm_nt_fused(x8, w8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = block(f, *operands), f.gemm_nt_fused(x8, w8)
            graphs.append(g)
            outs.append(out)
    for step in range(3):
        for t, new in zip(operands, block_operands(130, 256, 344, seed=20 + step)):
            t.copy_(new)
        want, want8 = block(f, *operands), f.gemm_nt_fused(x8, w8)
        torch.cuda.synchronize()
        for g, out in zip(graphs, outs):
            for t in out[0]:
                t.fill_(1.0)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out[0], want)) and torch.equal(out[1], want8)


def test_repeated_calls_agree(f):
    x, wg, wu, wd, dy = block_operands(513, 264, 1000)
    first = block(f, x, wg, wu, wd, dy)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(block(f, x, wg, wu, wd, dy), first))


def test_fp8_block(f):
    """A serving block: the gated product, its output quantised per token, the down projection added to the residual."""
    for T in (1, 30, 200):
        D, H = 256, 704
        x = rand(1, T, D)
        ws = [rand(s, *shape, std=shape[1] ** -0.5) for s, shape in ((2, (H, D)), (3, (H, D)), (4, (D, H)))]

        def quantise(t):
            s = t.float().abs().amax(dim=1).clamp(min=1e-6) / 448
            return (t.float() / s[:, None]).to(E4), s

        (xq, sx), (g, sg), (u, su), (d, sd) = (quantise(t) for t in (x, *ws))
        h = f.gated_nt(xq, g, u, sx, sg, su)
        _, _, v, tight, hw = F.gated_reference(xq, g, u, sx, sg, su)
        F.check(h, v, tight, hw, D, "gate and up")
        hq, sh = quantise(h)
        y = f.gemm_nt_fused(hq, d, sh, sd, residual=x)
        _, v, tight, hw = F.fused_reference(hq, d, sh, sd, res=x)
        F.check(y, v, tight, hw, H, "down")


def test_long_offsets(f):
    """Outputs, residuals and pre-activations past 2^32 bytes and 2^31 elements."""
    M, N, K = 70000, 32768, 16
    a, b = rand(1, M, K), rand(2, N, K)
    rows = torch.tensor([0, 1, 32767, 65535, 65536, M - 1], device=DEV)
    res = torch.zeros(M, N, dtype=BF, device=DEV)
    res[rows] = rand(3, len(rows), N)
    pre = torch.empty(M, N, device=DEV)
    out = f.gemm_nt_bf16_fused(a, b, activation="silu", residual=res, preact=pre)
    z, v, tight, hw = F.fused_reference(a[rows], b, name="silu", res=res[rows])
    F.check(out[rows], v, tight, hw, K, "rows")
    assert ((pre[rows].cpu().double() - z).abs() <= tight + hw).all()
    del res, out
    G = torch.zeros(M, N, dtype=BF, device=DEV)
    G[rows] = rand(4, len(rows), N)
    ga, gb, gbias = f.gemm_nt_bf16_fused_backward(G, a, b, "silu", pre, bias_grad=True)
    g64 = G[rows].cpu().double()
    dz = g64 * F.act("silu", z)[1]
    err = g64.abs() * (0.8 * (tight + hw) + 2.0 ** -19 * (1 + z.abs()))
    F.check(ga[rows], *F.backward_products(dz, err, b), N, "grad_a")
    F.check(gb, *F.backward_products(dz.t(), err.t(), a[rows]), 64, "grad_b")
    assert ((gbias.cpu().double() - dz.sum(0)).abs() <= err.sum(0) + 1e-5 * dz.abs().sum(0)).all()


def test_refusals_on_the_gpu(f):
    a, b = rand(1, 4, 32), rand(2, 8, 32)
    cpu = torch.zeros(8, 32, dtype=BF)
    with pytest.raises(ValueError, match="one GPU"):
        f.gemm_nt_bf16_fused(a, cpu)
    with pytest.raises(ValueError, match="residual"):
        f.gemm_nt_bf16_fused(a, b, residual=rand(3, 4, 9))
    with pytest.raises(ValueError, match="out"):
        f.gemm_nt_bf16_fused(a, b, out=torch.empty(4, 8, device=DEV))
    with pytest.raises(ValueError, match="preact"):
        f.gemm_nt_bf16_fused_backward(rand(3, 4, 8), a, b, activation="silu")
    with pytest.raises(ValueError, match="preact"):
        f.gated_nt_bf16(a, b, b, preact=torch.empty(4, 8, device=DEV))
    with pytest.raises(ValueError, match="bias"):
        f.gemm_nt_bf16_fused(a, b, bias=torch.zeros(1, device=DEV))
    with pytest.raises(f.Fp8GemmError):
        f.gemm_nt_bf16_fused(rand(1, 4, 12), rand(2, 8, 12))
    with pytest.raises(f.Fp8GemmError):
        f.gemm_nt_bf16_fused(strided(a, 4), b)
    with pytest.raises(ValueError, match="length"):
        f.gated_nt(rand(1, 4, 32, dtype=E5), rand(2, 8, 32, dtype=E4), rand(3, 8, 32, dtype=E4),
                   scale_gate=torch.ones(8, device=DEV), scale_up=torch.ones(1, device=DEV))
