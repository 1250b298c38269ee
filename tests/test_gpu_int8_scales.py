"""Integer products whose scales lie near the ends of FP32: an output within FP32
is finite whatever a sum times one of its scales alone would be.  Every build of
the dense and the ragged product, against exact references (tests/_experts.py).

The bound is that of tests/_experts.py, and half the smallest BF16 step, 2^-134,
where an output is below the normal numbers (rounded to FP32 and then to BF16:
twice that).
"""
import pytest
import torch

from tests import _experts as E
from tests import test_gpu_experts as X
from tests import test_gpu_int8 as D
from tests._experts import BF, DEV, codes, rand
from tests.test_gpu_experts import columns, f  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -133
# (row scales, channel scales), taken in turn: the product of any two and a sum stays within FP32
SETS = [((1.1 * 2.0 ** -10, 1.7 * 2.0 ** 90, 1.0 * 2.0 ** 96, 1.1 * 2.0 ** 97, -1.9 * 2.0 ** 120, 1.99 * 2.0 ** 127),
         (1.3 * 2.0 ** -110, 1.7 * 2.0 ** -112, -1.1 * 2.0 ** -115)),
        ((3 * 2.0 ** -149, 1.5 * 2.0 ** -130, -1.9 * 2.0 ** -110, 2.0 ** -60), (1.3 * 2.0 ** 20, -1.7 * 2.0 ** 30, 1.5 * 2.0 ** 75))]


def cycle(values, *shape):
    n = 1
    for s in shape:
        n *= s
    return torch.tensor([values[i % len(values)] for i in range(n)], dtype=torch.float32).view(*shape).to(DEV)


def check_dense(f, M, N, K, scales, bias=False, act="none"):  # noqa: F811
    a, b = codes(M + K, M, K), codes(N + 7 * K, N, K)
    a[M // 2] = 0                                          # sums of zero as well
    sa, sb = cycle(scales[0], M), cycle(scales[1], N)
    bv = rand(3, N, dtype=torch.float32) if bias else None
    got = f.gemm_nt_int8(a, b, sa, sb, bias=bv, activation=act)
    cols = columns(N)
    z = E.int_product(a, b[cols], sa, sb[cols])
    S = z.abs()
    if bias:
        z, S = z + bv[cols].cpu().double(), S + bv[cols].cpu().double().abs()
    v = z.clamp(min=0) if act == "relu" else z
    E.check_int(got[:, cols], z, S, f"{M}x{N}x{K}", v, TINY)


@pytest.mark.parametrize("scales", SETS, ids=["large", "small"])
@pytest.mark.parametrize("direct", [True, False], ids=["direct", "staged"])
@pytest.mark.parametrize("build", D.BUILDS, ids=lambda b: "-".join(map(str, b)))
def test_dense(f, build, direct, scales):  # noqa: F811
    size = D.builds(direct)[build]
    check_dense(f, *size, scales)
    check_dense(f, *size, scales, bias=True, act="none" if direct else "relu")


@pytest.mark.parametrize("scales", SETS, ids=["large", "small"])
@pytest.mark.parametrize("build", [b[1:] for b in X.BUILDS if b[0] == "int8"], ids=lambda b: "-".join(map(str, b)))
def test_ragged(f, build, scales):  # noqa: F811
    m, n, k, g = X.builds(X.OPS["int8"])[build]
    counts = E.divide(m, g, seed=m + n + k + g)
    a, b = codes(1, m, k), codes(2, g, n, k)
    sa, sb = cycle(scales[0], m), cycle(scales[1], g, n)
    out = f.grouped_gemm_ragged_int8(a, b, E.offsets_of(counts), sa, sb)
    cols = columns(n)
    for e, lo, hi in E.spans(counts):
        z = E.int_product(a[lo:hi], b[e][cols], sa[lo:hi], sb[e][cols])
        E.check_int(out[lo:hi][:, cols], z, z.abs(), f"expert {e}", None, TINY)


@pytest.mark.parametrize("M", [3, 300, 2500])
def test_past_the_largest(f, M):  # noqa: F811
    """Outputs past the largest number are infinities of their sign, and no others are."""
    a, b = codes(1, M, 144), codes(2, 136, 144)
    sa, sb = cycle((1.0, 2.0 ** 100, 1.5 * 2.0 ** 112, 2.0 ** 126), M), cycle((1.0, 2.0 ** -6), 136)
    z = E.int_product(a, b, sa, sb)
    got = f.gemm_nt_int8(a, b, sa, sb).cpu().double()
    # the largest BF16 number is 2^128 - 2^120; from half a step above it on, values round to an infinity
    over = z.abs() >= 2.0 ** 128 - 2.0 ** 119 + 2.0 ** 107
    under = z.abs() < 2.0 ** 128 - 2.0 ** 119 - 2.0 ** 107
    assert over.any() and under.any()
    assert (got[over] == z[over].sign() * float("inf")).all() and got[under].isfinite().all()


@pytest.mark.parametrize("M", [3, 300])
def test_quantised_from_large_values(f, M):  # noqa: F811
    """Rows up to the largest BF16 numbers, quantised, times weights small enough for finite outputs."""
    N, K = 136, 1040
    x = (rand(1, M, K, dtype=torch.float32) * 2.0 ** 122).to(BF)
    x[0] = x[0] * 2.0 ** -20
    q, s = f.quantize_rows_int8(x)
    assert float(s.max()) > 2.0 ** 115
    w, sw = codes(2, N, K), cycle((2.0 ** -30, 1.7 * 2.0 ** -25), N)
    z = E.int_product(q, w, s, sw)
    got = f.gemm_nt_int8(q, w, s, sw)
    E.check_int(got, z, z.abs(), "dense")
    ragged = f.grouped_gemm_ragged_int8(q, w[None], E.offsets_of([M]), s, sw[None])
    E.check_int(ragged, z, z.abs(), "ragged")
