"""Plain 64-bit references and error bounds of the fused and gated products.

With eps = 2^-8 (half a BF16 step, relative) a forward output o of exact value
r satisfies

    |o - r| <= eps |r| + e,

e the error of the FP32 computation before the rounding.  A sum z carries
dz <= 1e-5 S (S = |scales| sum_k |a b| + |bias|) on random data, and never more
than dz_hw, which adds what the matrix cores cut from the products (the
allowances of tests/_parity.py).  As in those checks, elements may need dz_hw
only up to random_cap() of them.

Activations: |act'| <= 1.13 for every one of them, and the FP32 evaluation
(exponential, reciprocal, erfc: a few units in the last place, the exponent's
argument rounded to 2^-24 |z|) is within 2^-20 |act(z)| + 2^-22 |z act'(z)|,
below 2^-19 |z|.  So e = 1.2 dz + 2^-19 |z| (fused), and for the gated product
act(g) u: e = |u| (1.2 dg + 2^-19 |g|) + |act(g)| du.

The backward products take dz = G act'(z) rounded to BF16.  The reference
rounds its own 64-bit dz the same way, so that only the elements that lie
within their error of a rounding border may differ, by one step 2^-7 |dz|:
those enter the bound as such, every other one only through the product's own
sum.  |act''| <= 0.8 (gelu at 0), so the error of dz is
|G| (0.8 dz_hw + 2^-19 (1 + |z|)); relu's slope jumps, so an element with
|z| <= dz_hw may be off by |G|.
"""
import math

import numpy as np
import torch

from tests._parity import _bf16_group_weights, gpu_bits, group_exponent_weights, random_cap

EPS = 2.0 ** -8
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(name, z):
    """(act(z), act'(z)) in float64."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        v, dv = z, torch.ones_like(z)
    else:
        c = math.sqrt(8 / math.pi)
        v, dv = c * (z + 0.044715 * z ** 3), c * (1 + 0.134145 * z ** 2)
    s = torch.sigmoid(v)
    return z * s, s + z * s * torch.sigmoid(-v) * dv


def weights_of(t):
    """(group weights, group term) of one operand for the matrix cores' cut."""
    if t.dtype == torch.bfloat16:
        return torch.from_numpy(_bf16_group_weights(gpu_bits(t), 32))
    fmt = 0 if t.dtype == torch.float8_e4m3fn else 1
    return torch.from_numpy(group_exponent_weights(t.cpu().view(torch.uint8).numpy(), fmt))


def product(a, b):
    """A . B^T in float64 on the CPU, its S and the hardware bound of its error (a, b: FP8 or BF16)."""
    x, y = a.cpu().double(), b.cpu().double()
    K = x.shape[1]
    S = x.abs() @ y.abs().t()
    cut = (2.0 ** -18 if a.dtype == torch.bfloat16 else 2.0 ** -9) * (weights_of(a) @ weights_of(b).t())
    return x @ y.t(), S, cut + (max(K, 8) / 8.0) * 2.0 ** -24 * S


def scaled(p, sa, sb):
    """The same with scales (None = 1)."""
    f = torch.ones((), dtype=torch.float64)
    if sa is not None:
        f = f * sa.cpu().double().reshape(-1, 1)
    if sb is not None:
        f = f * sb.cpu().double().reshape(1, -1)
    z, S, hw = p
    return z * f, S * f.abs(), hw * f.abs()


def check(got, ref, tight, hw, K, what):
    """Every element within eps |ref| + tight, but random_cap() that may take eps |ref| + tight + hw."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, what
    err = (got - ref).abs()
    fine = err <= EPS * ref.abs() + tight
    bad = ~fine
    n = int(bad.sum())
    worst = bad & ~(err <= EPS * ref.abs() + tight + hw)
    if worst.any():
        i = tuple(int(v) for v in worst.nonzero()[0])
        raise AssertionError(f"{what}: {int(worst.sum())} of {worst.numel()} elements outside the bound; first {i}: got "
                             f"{got[i].item()!r}, want {ref[i].item()!r}, tight {float(tight[i])!r}, hw {float(hw[i])!r}")
    cap = random_cap(got.numel(), K)
    assert n <= cap, f"{what}: {n} elements need the hardware allowance, {cap} may"


def fused_reference(a, b, sa=None, sb=None, bias=None, name="none", res=None):
    """(z, value, tight, hw) of the forward product."""
    z, S, hw = scaled(product(a, b), sa, sb)
    if bias is not None:
        z = z + bias.cpu().double()
        S = S + bias.cpu().double().abs()
    v, _ = act(name, z)
    tight = 1.2e-5 * S + 2.0 ** -19 * z.abs()
    if res is not None:
        r = res.cpu().double()
        v = v + r
        tight = tight + 2.0 ** -24 * r.abs()
    return z, v, tight, 1.2 * hw


def gated_reference(a, wg, wu, sa=None, sg=None, su=None, name="silu"):
    """(g, u, value, tight, hw) of the gated forward product."""
    g, Sg, hg = scaled(product(a, wg), sa, sg)
    u, Su, hu = scaled(product(a, wu), sa, su)
    v, _ = act(name, g)
    tight = u.abs() * (1.2e-5 * Sg + 2.0 ** -19 * g.abs()) + v.abs() * 1e-5 * Su
    hw = u.abs() * 1.2 * hg + v.abs() * hu + 1.2 * hg * hu
    return g, u, v * u, tight, hw


def bf16_near(x, err):
    """BF16 of x and the size of what an error `err` before the rounding can move (2^-7 |x| where it crosses a border)."""
    r = x.to(torch.bfloat16).double()
    moved = (x - err).to(torch.bfloat16) != (x + err).to(torch.bfloat16)
    return r, torch.where(moved, 2.0 ** -7 * x.abs() + err, torch.zeros_like(x))


def backward_products(dz, dz_err, other):
    """(ref, tight, hw) of dz . other with dz rounded to BF16, `other` BF16."""
    r, moved = bf16_near(dz, dz_err)
    o = other.cpu().double()
    S = r.abs() @ o.abs()
    cut = 2.0 ** -18 * (torch.from_numpy(_bf16_group_weights(gpu_bits(r.bfloat16()), 32)) @
                        torch.from_numpy(_bf16_group_weights(gpu_bits(other.t()), 32)).t())
    return r @ o, 1e-5 * S + moved @ o.abs(), cut + (max(dz.shape[1], 8) / 8.0) * 2.0 ** -24 * S
