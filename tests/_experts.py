"""Ragged groups of rows, and 64-bit references with error bounds of the
experts' products, the products in 8-bit integers and the quantisation.

BF16: the bounds of tests/_fused.py.  8-bit integers: the sums are exact, so an
output of exact value r is off by half a BF16 step, 2^-8 |r|, and by the FP32
operations before it, each of which rounds to 2^-24 of its result: the sum's
conversion and two scales (3 of |z|), the bias (|z + bias|, whose terms' errors
may exceed it where they cancel: 4 of S = |z| + |bias| together), the activation
(2^-19 |z|, and slopes up to 1.13, as in tests/_fused.py) and the residual.
"""
import torch

from tests import _fused as F

BF, DEV = torch.bfloat16, "cuda:0"


def rand(seed, *shape, dtype=BF, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def codes(seed, *shape):
    """Codes over the whole range, -128 included."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8).to(DEV)


def factors(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return ((torch.rand(*shape, generator=g) + 0.5) * 2e-3).to(DEV)


def offsets_of(counts, lead=0):
    """int32 offsets on the GPU of experts with these rows, the first after `lead` rows of none."""
    ends = torch.tensor([lead] + list(counts), dtype=torch.int64).cumsum(0)
    return ends.to(torch.int32).to(DEV)


def divide(rows, G, seed):
    """`rows` rows divided unevenly among G experts, about one in four of them without any."""
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(G, generator=g) ** 2 * (torch.rand(G, generator=g) > 0.25)
    if float(share.sum()) == 0:
        share[0] = 1
    cuts = torch.round(share.cumsum(0) / share.sum() * rows).long().tolist()
    return [b - a for a, b in zip([0] + cuts[:-1], cuts)]


def spans(counts, lead=0):
    """(expert, first row, end) of the experts that have rows."""
    at = lead
    for g, n in enumerate(counts):
        if n:
            yield g, at, at + n
        at += n


def with_nan_outside(t, counts, lead):
    """The rows of no expert hold NaN."""
    t[:lead] = float("nan")
    t[lead + sum(counts):] = float("nan")
    return t


def check_rows(got, a, b, counts, lead, cols, what):
    """The BF16 forward product's rows of every expert, in the given columns."""
    for g, lo, hi in spans(counts, lead):
        w = b[g][cols]
        z, S, hw = F.product(a[lo:hi], w)
        F.check(got[lo:hi][:, cols], z, 1e-5 * S, hw, a.shape[1], f"{what}, expert {g}")


def check_int(got, z, S, what, v=None, extra=0.0):
    """Integer products: z the exact value before the activation, v after it (None: z)."""
    r = z if v is None else v
    err = (got.detach().cpu().double() - r).abs()
    tol = F.EPS * r.abs() + 1.2 * 4 * 2.0 ** -24 * S + extra
    bad = ~(err <= tol * (1 + 2.0 ** -8))              # (the rounding is of the value with its error)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements outside the bound; first {i}: got "
                             f"{got[i].item()!r}, want {r[i].item()!r}, tolerance {float(tol[i])!r}")


def int_product(a, b, sa=None, sb=None):
    """sa sb (A . B^T), exact but for the 64-bit scales (|sum| < 2^31)."""
    z = a.cpu().double() @ b.cpu().double().t()
    if sa is not None:
        z = z * sa.cpu().double().reshape(-1, 1)
    if sb is not None:
        z = z * sb.cpu().double().reshape(1, -1)
    return z


def quantised(x):
    """(codes, scales) of the rows of a finite BF16 matrix, in 64 bits: the quotient of 8-bit significands is a half or
    at least 2^-18 away from one, so its 64-bit rounding decides rightly."""
    x = x.cpu().double()
    most = x.abs().amax(dim=1)
    q = x * 127 / torch.where(most > 0, most, torch.ones_like(most)).unsqueeze(1)
    return torch.round(q).to(torch.int8), most / 127
