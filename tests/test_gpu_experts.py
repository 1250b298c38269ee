"""Products over ragged groups of rows, BF16 with the backward pass and in 8-bit
integers, against 64-bit references (tests/_experts.py, tests/_fused.py).

The groups end anywhere in a tile, are empty, hold one row or all of them; rows
of no expert hold NaN and must neither be read nor written.
"""
import functools

import pytest
import torch

from tests import _experts as E
from tests import _fused as F
from tests._experts import BF, DEV, codes, factors, offsets_of, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def f():
    import fp8_gemm_amd
    fp8_gemm_amd.load_library()
    return fp8_gemm_amd


def columns(n, most=200):
    """Columns at both ends and around tile edges."""
    if n <= most:
        return torch.arange(n, device=DEV)
    keep = set(range(24)) | set(range(n - 40, n)) | {e + d for e in range(64, n, max(64, n // 16 // 64 * 64)) for d in (-1, 0)}
    return torch.tensor(sorted(keep), device=DEV)


def forward(f, kind, counts, N, K, lead=0, tail=0, seed=1):
    """One forward call checked; its operands."""
    M, G = lead + sum(counts) + tail, len(counts)
    offsets = offsets_of(counts, lead)
    out = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    cols = columns(N)
    if kind == "bf16":
        a = E.with_nan_outside(rand(seed, M, K), counts, lead)
        b = rand(seed + 1, G, N, K, std=0.25)
        assert f.grouped_gemm_ragged_bf16(a, b, offsets, out=out) is out
        E.check_rows(out, a, b, counts, lead, cols, f"{counts[:6]} {N}x{K}")
        rest = a, b, offsets
    else:
        a, b = codes(seed, M, K), codes(seed + 1, G, N, K)
        sa, sb = E.with_nan_outside(factors(seed + 2, M), counts, lead), factors(seed + 3, G, N)
        assert f.grouped_gemm_ragged_int8(a, b, offsets, sa, sb, out=out) is out
        for g, lo, hi in E.spans(counts, lead):
            z = E.int_product(a[lo:hi], b[g][cols], sa[lo:hi], sb[g][cols])
            E.check_int(out[lo:hi][:, cols], z, z.abs(), f"{counts[:6]} {N}x{K}, expert {g}")
        rest = a, b, offsets, sa, sb
    assert (out[:lead] == 7).all() and (out[lead + sum(counts):] == 7).all()
    return out, rest


COUNTS = [[1], [0, 1, 0], [5, 0, 16, 17, 1], [127, 1, 128, 129], [255, 257, 0, 64, 65], [0, 0, 0], [33, 600, 2],
          [3] * 70, [0] * 63 + [9, 40] + [0] * 70 + [150]]


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:5])) + f"x{len(c)}")
def test_forward(f, kind, counts):
    for N, K, lead, tail in ((8, 16, 0, 0), (136, 80, 3, 0), (264, 208, 0, 5), (40, 528, 130, 270)):
        forward(f, kind, counts, N, K, lead, tail)


def backward_check(f, a, b, offsets, counts, lead, seed=9, rows=None):
    """Both gradients checked (in a subset of the weight gradient's rows, of `rows` where given)."""
    M, K = a.shape
    G, N, _ = b.shape
    grad = E.with_nan_outside(rand(seed, M, N), counts, lead)
    ga, gb = f.grouped_gemm_ragged_bf16_backward(grad, a, b, offsets)
    end = lead + sum(counts)
    assert not ga[:lead].any() and not ga[end:].any()
    nc, kc = columns(N, 96), columns(K, 96)
    seen = set()
    for g, lo, hi in E.spans(counts, lead):
        seen.add(g)
        g6 = grad[lo:hi].cpu().double()
        zero = torch.zeros_like(g6)
        F.check(ga[lo:hi][:, kc], *F.backward_products(g6, zero, b[g][:, kc]), N, f"grad_a, expert {g}")
        F.check(gb[g][nc][:, kc], *F.backward_products(g6[:, nc.cpu()].t(), zero[:, nc.cpu()].t(), a[lo:hi][:, kc]), hi - lo, f"grad_b, expert {g}")
    for g in range(G):
        if g not in seen:
            assert not gb[g].any()
    return grad, ga, gb


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:5])) + f"x{len(c)}")
def test_backward(f, counts):
    for N, K, lead, tail in ((8, 8, 0, 0), (136, 72, 3, 0), (264, 208, 0, 5), (40, 520, 130, 270)):
        M = lead + sum(counts) + tail
        a = E.with_nan_outside(rand(1, M, K), counts, lead)
        b = rand(2, len(counts), N, K, std=0.25)
        backward_check(f, a, b, offsets_of(counts, lead), counts, lead)


# ---- every build, on sums that refill every ring slot, with whole and cut last K steps
OPS = {"bf16": 0, "int8": 1, "grad_a": 2, "grad_b": 3}


@functools.lru_cache(None)
def builds(op):
    """{build: the cheapest of the candidate sizes that takes it}."""
    import fp8_gemm_amd as f
    best = {}
    long = (1152, 1168) if op == 1 else ((576, 1024, 2832) if op == 3 else (576, 584))
    for m in (3, 17, 40, 100, 130, 200, 300, 500, 700, 1000, 1500, 2000, 3000, 5000, 9000):
        for x in (8, 24, 40, 64, 136, 264, 520, 1032, 2056, 4104, 8200):
            for red in long:
                for g in (1, 2, 4, 7, 16, 40, 70):
                    n, k = (red, x) if op == 2 else (x, red)
                    if op == 3 and m < 9 * 64 * g:
                        continue
                    p = f.experts_plan(op, m, n, k, g)
                    tail = op != 3 and p.variant != 4 and red == long[1]
                    key = (p.variant, p.tile_m, p.tile_n, tail)
                    cost = m * n * k + 20 * g * n * k
                    if cost < best.get(key, (1e300,))[0]:
                        best[key] = cost, (m, n, k, g)
    return {k: v[1] for k, v in best.items()}


TILES = [(7, 128, 128), (2, 128, 256), (1, 256, 256)]
FEW = [(4, 16 * cb, 16 * rb) for cb in (1, 2, 4) for rb in (1, 2, 4)]
BUILDS = [(kind, *t, tail) for kind in ("bf16", "int8", "grad_a") for t in TILES for tail in (False, True)] + \
         [(kind, *t, False) for kind in ("bf16", "int8") for t in FEW] + [("grad_b", *t, False) for t in TILES]


@pytest.mark.parametrize("build", BUILDS, ids=lambda b: "-".join(map(str, b)))
def test_every_build(f, build):
    kind = build[0]
    found = builds(OPS[kind])
    assert build[1:] in found, sorted(found)
    m, n, k, g = found[build[1:]]
    lead, tail = min(m // 20, 5), min(m // 10, 70)
    counts = E.divide(m - lead - tail, g, seed=m + n + k + g)
    if kind in ("bf16", "int8"):
        forward(f, kind, counts, n, k, lead, tail)
    else:
        a = E.with_nan_outside(rand(1, m, k), counts, lead)
        backward_check(f, a, rand(2, g, n, k, std=0.25), offsets_of(counts, lead), counts, lead)


def test_only_these_builds_exist():
    for kind, op in OPS.items():
        assert set(builds(op)) == {b[1:] for b in BUILDS if b[0] == kind}, kind


def test_persistent_rounds(f):
    """More tiles than workgroups, empty experts among them: the copies ahead of the next tile, one K step and many."""
    counts = [0, 1, 700, 0, 129, 1500, 3, 0, 2000, 256]
    for N, K in ((8200, 16), (8200, 208)):
        assert f.experts_plan(0, 4700, N, K, 10).workgroups > 512
        forward(f, "bf16", counts, N, K, 50, 61)
        forward(f, "int8", counts, N, K, 50, 61)
    a = E.with_nan_outside(rand(1, 4700, 4104), counts, 50)
    backward_check(f, a, rand(2, 10, 1032, 4104, std=0.25), offsets_of(counts, 50), counts, 50)
    # more than 64 experts, whose offsets are read anew for every tile
    counts = E.divide(9000, 150, 5)
    forward(f, "bf16", counts, 2056, 64, 7, 9)
    a = rand(1, 9000, 2056)
    backward_check(f, a, rand(2, 150, 136, 2056, std=0.25), offsets_of(counts), counts, 0)


def test_gradients_past_the_caches(f):
    """Weight gradients above 256 MB, whose stores bypass the caches; rows and columns that end inside a tile."""
    counts, N, K = [0, 150, 1, 129, 20, 0, 64, 3, 5], 4104, 4088
    a = E.with_nan_outside(rand(1, sum(counts) + 9, K), counts, 4)
    b = torch.zeros(9, N, K, dtype=BF, device=DEV)
    b[:, ::37] = rand(2, 9, (N + 36) // 37, K)
    assert b.numel() * 2 > 256 << 20
    backward_check(f, a, b, offsets_of(counts, 4), counts, 4)


# ---- as they are used
def test_strided(f):
    """Rows and experts apart in memory, NaN between them; outputs as columns of a wider buffer."""
    counts, lead, N, K = [40, 0, 170, 3], 2, 136, 72
    M, G = 220, 4
    offsets = offsets_of(counts, lead)
    a, b, grad = rand(1, M, K), rand(2, G, N, K), rand(3, M, N)
    want = f.grouped_gemm_ragged_bf16(a, b, offsets)[lead:lead + 213]
    ga, gb = f.grouped_gemm_ragged_bf16_backward(grad, a, b, offsets)
    wa = torch.full((M, K + 24), float("nan"), dtype=BF, device=DEV)[:, :K]
    wb = torch.full((G, N + 5, K + 8), float("nan"), dtype=BF, device=DEV)[:, :N, :K]
    wg = torch.full((M, N + 8), float("nan"), dtype=BF, device=DEV)[:, :N]
    for w, t in ((wa, a), (wb, b), (wg, grad)):
        w.copy_(t)
    buf = torch.full((M, N + 16), 7.0, dtype=BF, device=DEV)
    got = f.grouped_gemm_ragged_bf16(wa, wb, offsets, out=buf[:, 8:8 + N])
    assert torch.equal(got[lead:lead + 213], want) and (buf[:, :8] == 7).all() and (buf[:, 8 + N:] == 7).all()
    ga2, gb2 = f.grouped_gemm_ragged_bf16_backward(wg, wa, wb, offsets)
    assert torch.equal(ga, ga2) and torch.equal(gb, gb2)
    # every second expert of a larger set (the two halves of a merged gate and up projection)
    both = rand(4, G, 2 * N, K)
    up = f.grouped_gemm_ragged_bf16(a, both[:, N:], offsets)
    assert torch.equal(up[lead:lead + 213], f.grouped_gemm_ragged_bf16(a, both[:, N:].contiguous(), offsets)[lead:lead + 213])
    a8, b8 = codes(1, M, 80), codes(2, G, N, 80)
    wa8, wb8 = torch.zeros(M, 112, dtype=torch.int8, device=DEV)[:, :80], torch.zeros(G, N + 1, 96, dtype=torch.int8, device=DEV)[:, :N, :80]
    wa8.copy_(a8)
    wb8.copy_(b8)
    assert torch.equal(f.grouped_gemm_ragged_int8(wa8, wb8, offsets)[lead:lead + 213],
                       f.grouped_gemm_ragged_int8(a8, b8, offsets)[lead:lead + 213])


def test_gradients_on_request(f):
    counts = [30, 100, 0]
    a, b, grad, offsets = rand(1, 130, 64), rand(2, 3, 48, 64), rand(3, 130, 48), offsets_of(counts)
    ga, gb = f.grouped_gemm_ragged_bf16_backward(grad, a, b, offsets)
    only_a, none = f.grouped_gemm_ragged_bf16_backward(grad, a, b, offsets, b_grad=False)
    assert none is None and torch.equal(only_a, ga)
    none, only_b = f.grouped_gemm_ragged_bf16_backward(grad, a, b, offsets, a_grad=False)
    assert none is None and torch.equal(only_b, gb)
    assert f.grouped_gemm_ragged_bf16_backward(grad, a, b, offsets, a_grad=False, b_grad=False) == (None, None)


def test_empty_sizes(f):
    z = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
    assert f.grouped_gemm_ragged_bf16(z(0, 16), z(2, 8, 16), offsets_of([0, 0])).shape == (0, 8)
    assert f.grouped_gemm_ragged_bf16(z(5, 16), z(0, 8, 16), offsets_of([])).shape == (5, 8)
    assert f.grouped_gemm_ragged_bf16(z(5, 16), z(2, 0, 16), offsets_of([2, 3])).shape == (5, 0)
    for M, counts in ((5, [2, 3]), (1000, [300, 700])):
        # K = 0: the empty sum, in the experts' rows
        out = torch.full((M + 1, 8), 7.0, dtype=BF, device=DEV)
        f.grouped_gemm_ragged_bf16(z(M + 1, 0), z(2, 8, 0), offsets_of(counts), out=out)
        assert not out[:M].any() and (out[M] == 7).all()
        out.fill_(7.0)
        f.grouped_gemm_ragged_int8(z(M + 1, 0).to(torch.int8), z(2, 8, 0).to(torch.int8), offsets_of(counts), out=out)
        assert not out[:M].any() and (out[M] == 7).all()
    # gradients: no rows, no experts, no columns
    ga, gb = f.grouped_gemm_ragged_bf16_backward(z(0, 8), z(0, 16), rand(1, 3, 8, 16), offsets_of([0, 0, 0]))
    assert ga.shape == (0, 16) and not gb.any()
    ga, gb = f.grouped_gemm_ragged_bf16_backward(rand(1, 6, 8), rand(2, 6, 16), z(0, 8, 16), offsets_of([]))
    assert not ga.any() and gb.shape == (0, 8, 16)
    ga, gb = f.grouped_gemm_ragged_bf16_backward(z(6, 0), rand(2, 6, 16), z(2, 0, 16), offsets_of([2, 4]))
    assert not ga.any() and gb.shape == (2, 0, 16)


def test_one_expert_is_the_dense_product(f):
    a, b = rand(1, 300, 136), rand(2, 1, 264, 136)
    want = f.gemm_nt_bf16_fused(a, b[0])
    assert torch.equal(f.grouped_gemm_ragged_bf16(a, b, offsets_of([300])), want)
    a8, b8, sa, sb = codes(1, 300, 144), codes(2, 1, 264, 144), factors(3, 300), factors(4, 1, 264)
    assert torch.equal(f.grouped_gemm_ragged_int8(a8, b8, offsets_of([300]), sa, sb), f.gemm_nt_int8(a8, b8[0], sa, sb[0]))
    # without scales
    assert torch.equal(f.grouped_gemm_ragged_int8(a8, b8, offsets_of([300])), f.gemm_nt_int8(a8, b8[0]))


@pytest.mark.parametrize("M,N,K", [(60, 64, 32), (900, 136, 200)])
def test_bad_offsets_stay_inside(f, M, N, K):
    """Offsets outside 0 .. M or decreasing: no fault, and nothing written outside the rows that some reading of them gives."""
    buf = torch.full((M + 64, N), 7.0, dtype=BF, device=DEV)
    out = buf[32:32 + M]
    a, b = rand(1, M, K), rand(2, 4, N, K)
    for offs in ([-5, 10, 20, 1 << 30, 2147483647], [-2147483648, 0, M + 7, M, M], [M, 20, 40, 10, 50], [40, 40, 5, 5, 3]):
        o = torch.tensor(offs, dtype=torch.int64).to(torch.int32).to(DEV)
        f.grouped_gemm_ragged_bf16(a, b, o, out=out)
        ga, gb = f.grouped_gemm_ragged_bf16_backward(out.clone(), a, b, o)
        torch.cuda.synchronize()
        assert (buf[:32] == 7).all() and (buf[32 + M:] == 7).all() and ga.shape == a.shape and gb.shape == b.shape
    # far more tiles than any offsets that do not decrease can make, in one batch of 64 experts and in several
    for G in (60, 200):
        many = torch.zeros(G, N, K, dtype=BF, device=DEV)
        o = torch.tensor([0, M] * (G // 2) + [0], dtype=torch.int32, device=DEV)
        f.grouped_gemm_ragged_bf16(a, many, o, out=out)
        ga, gb = f.grouped_gemm_ragged_bf16_backward(out.clone(), a, many, o)
        torch.cuda.synchronize()
        assert (buf[:32] == 7).all() and (buf[32 + M:] == 7).all()
    # values past either end count as that end
    o = torch.tensor([-5, 10, 20, 40, 2147483647], dtype=torch.int32, device=DEV)
    E.check_rows(f.grouped_gemm_ragged_bf16(a, b, o), a, b, [10, 10, 20, M - 40], 0, columns(N), "clamped")


def test_infinities_stay_with_their_row(f):
    counts, K, N = [20, 200, 9], 64, 72
    a, b, offsets = rand(1, 229, K), rand(2, 3, N, K), offsets_of([20, 200, 9])
    clean = f.grouped_gemm_ragged_bf16(a, b, offsets)
    bad = a.clone()
    bad[25, 3], bad[100, 7], bad[0, 0] = float("nan"), float("inf"), float("-inf")
    got = f.grouped_gemm_ragged_bf16(bad, b, offsets)
    same = torch.ones(229, dtype=torch.bool, device=DEV)
    same[[25, 100, 0]] = False
    assert torch.equal(got[same], clean[same])
    assert got[25].isnan().all() and not got[100].isfinite().any() and not got[0].isfinite().any()
    # a weight gradient holds what its expert's rows hold, and no other's
    grad = rand(3, 229, N)
    _, gb = f.grouped_gemm_ragged_bf16_backward(grad, a, b, offsets)
    _, gb2 = f.grouped_gemm_ragged_bf16_backward(grad, bad, b, offsets)
    assert torch.equal(gb[2], gb2[2]) and gb2[1][:, 3].isnan().all() and not gb2[0][:, 0].isfinite().any()
    assert torch.equal(gb[1][:, 8:], gb2[1][:, 8:])


def layer(f, x, w1, w2, offsets, dy):
    """Two expert products in a row, forward and backward."""
    h = f.grouped_gemm_ragged_bf16(x, w1, offsets)
    y = f.grouped_gemm_ragged_bf16(h, w2, offsets)
    dh, dw2 = f.grouped_gemm_ragged_bf16_backward(dy, h, w2, offsets)
    dx, dw1 = f.grouped_gemm_ragged_bf16_backward(dh, x, w1, offsets)
    return y, dx, dw1, dw2


def layer_operands(counts, D, H, seed=1):
    T, G = sum(counts), len(counts)
    return rand(seed, T, D), rand(seed + 1, G, H, D, std=D ** -0.5), rand(seed + 2, G, D, H, std=H ** -0.5), offsets_of(counts), rand(seed + 3, T, D)


@pytest.mark.parametrize("counts,D,H", [([1, 0, 2], 64, 160), ([50, 3, 0, 150], 136, 344), ([700, 333], 256, 680)])
def test_expert_layer(f, counts, D, H):
    ops = layer_operands(counts, D, H)
    got = layer(f, *ops)
    x, w1, w2, dy = (ops[i].cpu().double() for i in (0, 1, 2, 4))
    want = [torch.zeros(x.shape[0], D, dtype=torch.float64), torch.zeros_like(x), torch.zeros_like(w1), torch.zeros_like(w2)]
    for g, lo, hi in E.spans(counts):
        h = x[lo:hi] @ w1[g].t()
        dh = dy[lo:hi] @ w2[g]
        want[0][lo:hi], want[1][lo:hi] = h @ w2[g].t(), dh @ w1[g]
        want[2][g], want[3][g] = dh.t() @ x[lo:hi], dy[lo:hi].t() @ h
    # at most two roundings of eps in a row
    for a, b, name in zip(got, want, ("y", "dx", "dw1", "dw2")):
        rel = float((a.cpu().double() - b).norm() / b.norm())
        assert rel <= 2 * F.EPS, (name, rel)


def test_gradients_against_differences(f):
    """<grad, direction> against central differences of sum(G * out) in 64 bits."""
    counts, N, K, h = [30, 0, 41], 72, 80, 1e-5
    a, b, G, offsets = rand(1, 71, K), rand(2, 3, N, K, std=0.1), rand(3, 71, N), offsets_of(counts)
    grads = f.grouped_gemm_ragged_bf16_backward(G, a, b, offsets)
    at = [a.cpu().double(), b.cpu().double()]
    G6 = G.cpu().double()

    def loss(x, w):
        return sum((G6[lo:hi] * (x[lo:hi] @ w[g].t())).sum() for g, lo, hi in E.spans(counts))

    for i, grad in enumerate(grads):
        d = torch.randn(at[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        up = loss(*(t + h * d if k == i else t for k, t in enumerate(at)))
        down = loss(*(t - h * d if k == i else t for k, t in enumerate(at)))
        g6 = grad.cpu().double()
        # each entry off by one rounding, in directions that do not depend on d: six standard deviations of their sum
        tol = 6 * F.EPS * float((g6 * d).norm()) + 1e-4 * abs(float(up - down)) / (2 * h)
        assert abs(float((g6 * d).sum()) - float(up - down) / (2 * h)) <= tol, i


def serve(f, x, w1, s1, w2, s2, offsets):
    """The same layer in 8-bit integers, its activations quantised in between."""
    q, sx = f.quantize_rows_int8(x)
    h = f.grouped_gemm_ragged_int8(q, w1, offsets, sx, s1)
    qh, sh = f.quantize_rows_int8(h)
    return q, sx, h, qh, sh, f.grouped_gemm_ragged_int8(qh, w2, offsets, sh, s2)


def serve_operands(counts, D, H, seed=1):
    T, G = sum(counts), len(counts)
    return (rand(seed, T, D), codes(seed + 1, G, H, D), factors(seed + 2, G, H), codes(seed + 3, G, D, H), factors(seed + 4, G, D), offsets_of(counts))


@pytest.mark.parametrize("counts,D,H", [([1], 64, 160), ([1, 0, 7], 256, 704), ([40, 0, 130, 300], 128, 336)])
def test_integer_layer(f, counts, D, H):
    x, w1, s1, w2, s2, offsets = serve_operands(counts, D, H)
    q, sx, h, qh, sh, y = serve(f, x, w1, s1, w2, s2, offsets)
    for inp, qq, s in ((x, q, sx), (h, qh, sh)):
        want, scale = E.quantised(inp)
        assert torch.equal(qq.cpu(), want) and ((s.cpu().double() - scale).abs() <= 2.0 ** -24 * scale).all()
    for qq, s, w, sw, out in ((q, sx, w1, s1, h), (qh, sh, w2, s2, y)):
        for g, lo, hi in E.spans(counts):
            z = E.int_product(qq[lo:hi], w[g], s[lo:hi], sw[g])
            E.check_int(out[lo:hi], z, z.abs(), f"expert {g}")


def test_streams(f):
    """Two streams at once, each with its own operands, against the same calls one after the other."""
    train = [layer_operands([100, 0, 201, 50], 128, 344, seed=10 * s) for s in range(2)]
    ints = [serve_operands([3, 0, 30], 256, 512, seed=10 * s) for s in range(2)]
    want = [(layer(f, *t), serve(f, *i)) for t, i in zip(train, ints)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((layer(f, *train[i]), serve(f, *ints[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for x, y in zip(r[0] + r[1], want[i][0] + want[i][1]):
                assert torch.equal(x, y)


def test_graphs(f):
    """Two captured steps replayed in turn with eager work between, on new values and new offsets: a captured step
    takes the rows that the offsets give when it is replayed."""
    splits = [[60, 0, 70], [0, 130, 0], [1, 2, 127]]
    t, i = layer_operands(splits[0], 128, 344), serve_operands(splits[0], 128, 352)
    layer(f, *t), serve(f, *i)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = layer(f, *t) + serve(f, *i)
            graphs.append(g)
            outs.append(out)
    for step, counts in enumerate(splits):
        for old, new in zip(t + i, layer_operands(counts, 128, 344, seed=30 + step) + serve_operands(counts, 128, 352, seed=60 + step)):
            old.copy_(new)
        want = layer(f, *t) + serve(f, *i)
        torch.cuda.synchronize()
        for g, out in zip(graphs, outs):
            for o in out:
                o.fill_(1)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_repeated_calls_agree(f):
    t, i = layer_operands([300, 0, 129, 84], 264, 1000), serve_operands([90, 8, 0, 33], 256, 1008)
    first = layer(f, *t) + serve(f, *i)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(layer(f, *t) + serve(f, *i), first))


def test_long_offsets(f):
    """Rows, outputs and weights past 2^32 bytes and 2^31 elements."""
    M, N, K, G = 70000, 32768, 16, 3
    counts = [30000, 0, M - 30000]
    a, b, offsets = rand(1, M, K), rand(2, G, N, K), offsets_of(counts)
    out = f.grouped_gemm_ragged_bf16(a, b, offsets)
    rows = torch.tensor([0, 1, 29999, 30000, 32767, 65535, 65536, M - 1], device=DEV)
    for r in rows.tolist():
        z, S, hw = F.product(a[r:r + 1], b[0 if r < 30000 else 2])
        F.check(out[r:r + 1], z, 1e-5 * S, hw, K, f"row {r}")
    grad = torch.zeros(M, N, dtype=BF, device=DEV)
    grad[rows] = rand(4, len(rows), N)
    ga, gb = f.grouped_gemm_ragged_bf16_backward(grad, a, b, offsets)
    for g, sel in ((0, rows[:3]), (2, rows[3:])):
        g6 = grad[sel].cpu().double()
        F.check(ga[sel], *F.backward_products(g6, torch.zeros_like(g6), b[g]), N, f"grad_a {g}")
        F.check(gb[g], *F.backward_products(g6.t(), torch.zeros_like(g6).t(), a[sel]), 64, f"grad_b {g}")
    assert not gb[1].any()
    del out, grad, ga, gb
    # the last expert's weights begin past 2^32 bytes
    G, N, K = 5, 2048, 262144
    a, offsets = rand(5, 40, K, std=0.1), offsets_of([7, 0, 9, 0, 24])
    b = torch.zeros(G, N, K, dtype=BF, device=DEV)
    part = rand(6, G, 64, K)
    b[:, -64:] = part
    out = f.grouped_gemm_ragged_bf16(a, b, offsets)
    for g, lo, hi in E.spans([7, 0, 9, 0, 24]):
        z, S, hw = F.product(a[lo:hi], part[g])
        F.check(out[lo:hi, -64:], z, 1e-5 * S, hw, K, f"expert {g}")
        assert not out[lo:hi, :-64].any()


def test_refusals_on_the_gpu(f):
    a, b, o = rand(1, 6, 32), rand(2, 2, 8, 32), offsets_of([2, 4])
    with pytest.raises(ValueError, match="one GPU"):
        f.grouped_gemm_ragged_bf16(a, b, o.cpu())
    with pytest.raises(ValueError, match="out"):
        f.grouped_gemm_ragged_bf16(a, b, o, out=torch.empty(6, 8, device=DEV))
    with pytest.raises(f.Fp8GemmError, match="overlap"):
        buf = torch.zeros(6, 64, dtype=BF, device=DEV)
        f.grouped_gemm_ragged_bf16(buf[:, :32], b, o, out=buf[:, 24:32])
    with pytest.raises(f.Fp8GemmError, match="overlap"):
        f.grouped_gemm_ragged_bf16(a, b, o, out=b[0, :6, :8])
    with pytest.raises((f.Fp8GemmError, ValueError)):
        f.grouped_gemm_ragged_bf16_backward(rand(3, 1, 8).expand(6, 8), a, b, o)
    with pytest.raises((f.Fp8GemmError, ValueError)):
        f.grouped_gemm_ragged_bf16(a, b[:1].expand(2, 8, 32), o)
