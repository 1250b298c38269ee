"""Activations and their slopes of the fused products far from zero, where an
absolute bound would hide them: relative bounds against 64 bits."""
import math

import pytest
import torch

from tests import _fused as F
from tests.test_gpu_fused import BF, DEV, E4, f  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu

OVERFLOW = 88.7                 # exp of more than 88.72 is infinite in FP32


def exponent(name, z):
    """The argument of the exponential that act and act' evaluate."""
    if name == "gelu":
        return z * z / 2
    return z if name == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)


@pytest.mark.parametrize("name,points", [
    ("silu", [-2.0, -5.5, -17.0, -29.0, -30.0, -31.0, -40.0, -60.5, -80.0, -87.0, -88.0, -88.6, -95.0, -99.0, -101.0,
              -500.0, -3e38, 20.0, 29.0, 31.0, 95.0, 3e38]),
    ("gelu", [-2.0, -5.5, -9.0, -12.5, 6.0, 13.0, 29.0, 31.0, 3e38]),
    ("gelu_tanh", [-2.0, -5.5, -8.0, -9.5, 6.0, 13.0, 29.0, 31.0, 3e38]),
])
def test_slopes_far_from_zero(f, name, points):
    """The bias gradient of one row whose output gradient is 1 is act'(z) itself, in FP32."""
    z = torch.tensor(points, device=DEV)
    n = len(points)
    one = torch.ones(1, n, dtype=BF, device=DEV)
    x, w = torch.zeros(1, 8, dtype=BF, device=DEV), torch.zeros(n, 8, dtype=BF, device=DEV)
    got = f.gemm_nt_bf16_fused_backward(one, x, w, name, z[None], bias_grad=True)[2].cpu().double()
    z64 = z.cpu().double()
    _, want = F.act(name, z64.clamp(-1e3, 1e3))
    # FP32 evaluation: the exponent's argument v is rounded to 2^-24 |v| a few times, every other step to 2^-24, none of
    # them amplified more than 2 times (1 + z (1 - s) at z = -2).  Past the exponential's overflow the sigmoid is 0, and
    # just before it a subnormal number: z times it is off by 2^-128 |z| and 2^-149 |z|.
    v = exponent(name, z64).abs().clamp(max=128)
    tol = 2.0 ** -20 * (1 + v) * want.abs() + 2.0 ** -149 * z64.abs().clamp(max=128)
    if name == "silu":
        tol = tol + torch.where(z64 < -OVERFLOW, 2.0 ** -128 * z64.abs().clamp(max=128), torch.zeros_like(z64))
    off = (got - want).abs()
    assert (off <= tol).all(), [(p, g, w) for p, g, w, bad in zip(points, got.tolist(), want.tolist(), off > tol) if bad]


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 100, 2100])
def test_small_sigmoids(f, name, M):
    """Sigmoids between 2^-128 and 2^-126, whose products with z are normal BF16 numbers."""
    v = torch.tensor([-87.0, -87.2, -87.4, -87.7, -88.0, -88.3, -88.6], dtype=torch.float64)
    z = v if name == "silu" else torch.linspace(-10.06, -9.98, 81, dtype=torch.float64)
    z = z.float().repeat(300)[:300]
    z64 = z.double()
    if name == "gelu_tanh":
        z64 = z64[exponent(name, z64) > -OVERFLOW]
        assert (exponent(name, z64) < -87.4).any()
    n = len(z64)
    bias = z64.float().to(DEV)
    want, _ = F.act(name, z64)
    # one rounding, and FP32: up to eight roundings of 2^-24 in the exponent's argument (the tanh form's polynomial, its
    # two constants, the factor log2 e), which is at most 89: 8 * 89 * 2^-24 < 2^-14
    tol = (F.EPS + 2.0 ** -14) * want.abs()
    x, w = torch.zeros(M, 16, device=DEV), torch.zeros(n, 16, device=DEV)
    for got in (f.gemm_nt_bf16_fused(x.to(BF), w.to(BF), bias=bias, activation=name),
                f.gemm_nt_fused(x.to(E4), w.to(E4), bias=bias, activation=name)):
        off = (got.cpu().double() - want).abs()
        assert (off <= tol).all(), (float(z64[(off > tol).any(0)][0]), int((off > tol).sum()))
