"""Products in 8-bit integers with a fused epilogue and the quantisation of rows,
against exact references (tests/_experts.py)."""
import functools

import pytest
import torch

from tests import _experts as E
from tests import _fused as F
from tests._experts import BF, DEV, codes, factors, rand
from tests.test_gpu_experts import FEW, TILES, columns, f  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu


def check(f, M, N, K, i, res=None, out=None):  # noqa: F811
    """One call with the i-th mix of scales, bias, activation and residual."""
    a, b = codes(M + K, M, K), codes(N + 7 * K, N, K)
    sa, sb = [factors(1, M), factors(1, 1), None][i % 3], [factors(2, N), None, factors(2, 1)][i % 3]
    if sa is None and sb is None:
        sb = factors(2, N)
    if i % 3 == 1:
        sa = sa * 1e-3
    bias = rand(3, N, dtype=torch.float32) if i % 2 else None
    if res is None and i not in (2, 5, 10):                # (5, 10: no activation either, the direct epilogue)
        res = rand(4, M, N)
    kept = None if res is None else res.clone()
    name = F.ACTS[i % 5]
    got = f.gemm_nt_int8(a, b, sa, sb, bias=bias, activation=name, residual=res, out=out)
    cols = columns(N)
    pick = lambda t: t if t is None or t.numel() == 1 else t[cols]  # noqa: E731
    z = E.int_product(a, b[cols], sa, pick(sb))
    S = z.abs()
    if bias is not None:
        z, S = z + pick(bias).cpu().double(), S + pick(bias).cpu().double().abs()
    v, _ = F.act(name, z)
    extra = 2.0 ** -19 * z.abs()
    if kept is not None:
        r = kept[:, cols].cpu().double()
        v, extra = v + r, extra + 2.0 ** -24 * (v.abs() + r.abs())
    E.check_int(got[:, cols], z, S, f"{name} {M}x{N}x{K}", v, extra)


SHAPES = [(1, 1, 16), (1, 130, 272), (5, 33, 400), (16, 64, 128), (17, 100, 144), (33, 257, 528), (64, 48, 1040),
          (65, 300, 272), (128, 256, 128), (130, 515, 400), (257, 260, 1168), (300, 1003, 144), (2100, 136, 80)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(f, M, N, K):  # noqa: F811
    for i in (0, 1, 2, 3, 4, 5, 10):
        check(f, M, N, K, i)


@functools.lru_cache(None)
def builds(direct):
    """{build: the cheapest of the candidate sizes that takes it}; direct: whole chunks of columns and neither activation
    nor residual."""
    import fp8_gemm_amd as f
    best = {}
    for m in (1, 3, 17, 40, 65, 130, 300, 700, 1000, 2000, 2100, 3000):
        for n in (8, 40, 136, 520, 1032, 2056, 4104, 8200, 14336):
            for k in (1152, 1168, 2048):
                p = f.experts_plan(4, m, n if direct else n - 3, k)
                key = (p.variant, p.tile_m, p.tile_n, p.variant != 4 and k % 128 != 0)
                if m * n * k < best.get(key, (1e300,))[0]:
                    best[key] = m * n * k, (m, n if direct else n - 3, k)
    return {k: v[1] for k, v in best.items()}


BUILDS = [(*t, tail) for t in TILES for tail in (False, True)] + [(*t, False) for t in FEW]


@pytest.mark.parametrize("direct", [True, False], ids=["direct", "staged"])
@pytest.mark.parametrize("build", BUILDS, ids=lambda b: "-".join(map(str, b)))
def test_every_build(f, build, direct):  # noqa: F811
    found = builds(direct)
    assert build in found, sorted(found)
    for i in (5, 10) if direct else (3, 2):
        check(f, *found[build], i)


def test_only_these_builds_exist():
    assert set(builds(True)) == set(builds(False)) == set(BUILDS)


def test_persistent_rounds(f):  # noqa: F811
    """More tiles than workgroups: the copies ahead of the next tile, with and without a K tail, one step and many."""
    for M, N, K in ((4100, 8200, 16), (4100, 8200, 144), (4100, 8200, 400), (9000, 5000, 16), (20000, 1032, 272)):
        assert f.experts_plan(4, M, N, K).workgroups > 300
        check(f, M, N, K, 5)


@pytest.mark.parametrize("M", [1, 40, 200, 2100])
def test_sums_are_exact(f, M):  # noqa: F811
    """Sums at the ends of 32 bits and sums of +-1, where FP32 adds would lose the last units."""
    K, N = 131056, 24
    a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    b = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    b[1], b[2, :K // 2] = 127, 127
    b[3].zero_()
    b[3, -1] = 1
    b[4, 0] = 127
    s = torch.full((1,), 2.0 ** -20, device=DEV)
    z = E.int_product(a[:1], b, s)
    got = f.gemm_nt_int8(a, b, s)
    E.check_int(got, z.expand(M, N), z.abs().expand(M, N), "ends")
    # a difference of one unit of 2^30: exact after the other terms cancel
    a.fill_(127)
    b.zero_()
    b[:, 0::2], b[:, 1::2] = 127, -127
    b[:, -1] = -126
    got = f.gemm_nt_int8(a, b)
    assert (got == 127).all()


def test_in_place_and_strided(f):  # noqa: F811
    for M, N, K in ((3, 37, 208), (70, 130, 272), (1500, 1030, 80)):
        buf = torch.full((M, (N + 7) // 8 * 8 + 8), 7.0, dtype=BF, device=DEV)
        res = buf[:, :N]
        res.copy_(rand(5, M, N))
        check(f, M, N, K, 0, res=res, out=res)
        assert (buf[:, N:] == 7).all()
        a, b = codes(1, M, K), codes(2, N, K)
        wa, wb = (torch.zeros(t.shape[0], K + 48, dtype=torch.int8, device=DEV)[:, :K] for t in (a, b))
        wa.copy_(a)
        wb.copy_(b)
        assert torch.equal(f.gemm_nt_int8(wa, wb), f.gemm_nt_int8(a, b))


def test_empty(f):  # noqa: F811
    z = lambda *s: torch.zeros(*s, dtype=torch.int8, device=DEV)  # noqa: E731
    assert f.gemm_nt_int8(z(0, 32), z(5, 32)).shape == (0, 5) and f.gemm_nt_int8(z(3, 32), z(0, 32)).shape == (3, 0)
    bias = rand(1, 40, dtype=torch.float32)
    for M in (3, 3000):
        assert torch.equal(f.gemm_nt_int8(z(M, 0), z(40, 0), bias=bias), bias.bfloat16().expand(M, 40))
    q, s = f.quantize_rows_int8(torch.zeros(0, 32, dtype=BF, device=DEV))
    assert q.shape == (0, 32) and s.shape == (0,)
    q, s = f.quantize_rows_int8(torch.zeros(3, 0, dtype=BF, device=DEV))
    assert q.shape == (3, 0) and not s.any()


# ---- quantisation
def check_quantised(f, x):  # noqa: F811
    q, s = f.quantize_rows_int8(x)
    want, scale = E.quantised(x)
    assert q.dtype == torch.int8 and s.dtype == torch.float32
    assert torch.equal(q.cpu(), want)
    # one rounding, or half the smallest FP32 step
    assert ((s.cpu().double() - scale).abs() <= 2.0 ** -24 * scale + 2.0 ** -150).all()
    return q, s


@pytest.mark.parametrize("M", [1, 3, 130, 600, 2050])
@pytest.mark.parametrize("K", [16, 48, 512, 528, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 14336, 16384, 16400])
def test_quantise(f, M, K):  # noqa: F811
    if M * K > 12_000_000:
        pytest.skip("covered by fewer rows")
    x = rand(M + K, M, K)
    x[:, ::64] *= 10
    x[M // 2] = 0
    check_quantised(f, x)


@pytest.mark.parametrize("M,K", [(2, 32768), (3, 32784), (1, 65536), (2, 65552), (2, 131056), (600, 16384), (520, 8208), (2100, 4096)])
def test_quantise_long_rows(f, M, K):  # noqa: F811
    check_quantised(f, rand(K, M, K))


def test_quantise_every_significand(f):  # noqa: F811
    """Every quotient of two 8-bit significands over 10 binades: all halves, to even, and all else to the nearest."""
    sig = torch.arange(128, 256, dtype=torch.float64)
    rows = []
    for d in range(10):
        rows.append((sig * 2.0 ** -d).unsqueeze(0).expand(128, 128))
    x = torch.cat(rows, dim=1)                             # [128, 1280]
    x = torch.cat((x, -x), dim=1)
    x = x * torch.where(x.abs() <= sig.unsqueeze(1), 1.0, 0.5)   # nothing above the row's largest
    x[:, 5] = sig
    for e in (0, -40, 60, -125, 100, 120):                 # up to the ends of the exponent, subnormal values among them
        y = (x * 2.0 ** e).to(BF).to(DEV)
        q, _ = check_quantised(f, y)
        assert int(q.max()) == 127 and int(q.min()) >= -127
    halves = 127 * x / sig.unsqueeze(1)
    assert int(((halves - halves.floor()) == 0.5).sum()) > 100


def test_quantise_smallest_and_largest(f):  # noqa: F811
    x = torch.zeros(6, 64, dtype=torch.float64)
    x[0, 3], x[0, 5] = 2.0 ** -133, -2.0 ** -133           # the smallest BF16 number
    x[1, 7], x[1, 8] = 3 * 2.0 ** -133, 2.0 ** -133
    x[2, 1], x[2, 2] = 255 * 2.0 ** 120, -2.0 ** -133      # the largest, and nothing beside it
    x[3, 1], x[3, 2] = 2.0 ** -126, 2.0 ** -127
    x[4] = 1.0
    check_quantised(f, x.to(BF).to(DEV))


@pytest.mark.parametrize("K", [64, 2064, 8192, 70000 // 16 * 16])
def test_quantise_not_finite(f, K):  # noqa: F811
    x = rand(1, 5, K)
    x[1, 3], x[2, K - 1], x[3, 0] = float("nan"), float("inf"), float("-inf")
    q, s = f.quantize_rows_int8(x)
    assert s[[1, 2, 3]].isnan().all() and not q[[1, 2, 3]].any()
    keep = x[[0, 4]]
    want, scale = f.quantize_rows_int8(keep)
    assert torch.equal(q[[0, 4]], want) and torch.equal(s[[0, 4]], scale)
    y = f.gemm_nt_int8(q, codes(2, 8, K), s)
    assert y[[1, 2, 3]].isnan().all() and y[[0, 4]].isfinite().all()


def test_quantise_strided(f):  # noqa: F811
    for M, K in ((5, 80), (300, 2064), (7, 4112)):
        x = rand(1, M, K)
        want = f.quantize_rows_int8(x)
        wide = torch.full((M, K + 24), float("inf"), dtype=BF, device=DEV)
        wide[:, :K] = x
        buf = torch.full((M, K + 32), 9, dtype=torch.int8, device=DEV)
        scales = torch.zeros(M, device=DEV)
        q, s = f.quantize_rows_int8(wide[:, :K], codes=buf[:, :K], scales=scales)
        assert s is scales and torch.equal(q, want[0]) and torch.equal(s, want[1]) and (buf[:, K:] == 9).all()
    with pytest.raises(f.Fp8GemmError, match="overlap"):
        f.quantize_rows_int8(x, codes=x.view(torch.int8)[:, :4112])
    with pytest.raises(f.Fp8GemmError, match="multiple"):
        f.quantize_rows_int8(torch.zeros(2, 24, dtype=BF, device=DEV))


def test_long_offsets(f):  # noqa: F811
    """Rows, codes and outputs past 2^32 bytes."""
    M, K = 140000, 32768
    x = torch.zeros(M, K, dtype=BF, device=DEV)
    rows = torch.tensor([0, 65535, 65536, 131072, M - 1], device=DEV)
    x[rows] = rand(1, len(rows), K)
    q, s = f.quantize_rows_int8(x)
    del x
    want, scale = f.quantize_rows_int8(rand(1, len(rows), K))
    assert torch.equal(q[rows], want) and torch.equal(s[rows], scale) and int((s != 0).sum()) == len(rows)
    b, sb = codes(2, 8, K), factors(3, 8)
    y = f.gemm_nt_int8(q, b, s, sb)
    assert torch.equal(y[rows], f.gemm_nt_int8(want, b, scale, sb))
    del q
    a, b = codes(4, M, 16), codes(5, K, 16)
    out = f.gemm_nt_int8(a, b)
    for r in rows.tolist():
        z = E.int_product(a[r:r + 1], b)
        E.check_int(out[r:r + 1], z, z.abs(), f"row {r}")
