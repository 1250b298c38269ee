"""The product with a fused epilogue and the gated feed-forward product, as they are measured.

Two operators, each with FP8 operands (serving) and BF16 operands (serving and training):

  fused   Z = sa[m] sb[n] (A . B^T) + bias[n],   D = act(Z) + R
          backward (BF16): dZ = dD act'(Z),  dA = dZ . B,  dB = dZ^T . A,  dbias = column sums of dZ
  gated   G = sa[m] sg[n] (A . Wg^T),  U = sa[m] su[n] (A . Wu^T),   H = act(G) U
          backward (BF16): dG = dH U act'(G),  dU = dH act(G),
          dA = dG . Wg + dU . Wu,  dWg = dG^T . A,  dWu = dU^T . A

A is [M, K] (tokens), B, Wg and Wu are [N, K] (weights), all K-contiguous.  A case names its operator (`op`), its
operands' types (`kind`: "e4m3", "e5m2", "mixed" for E5M2 tokens with E4M3 weights, "bf16"), whether it is a training
step (`train`: forward and backward, gradients returned) and its sizes.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    def fused(name, kind, m, n, k, act, bias, residual, train=False):
        return dict(name=name, op="fused", kind=kind, m=m, n=n, k=k, act=act, bias=bias, residual=residual, train=train)

    def gated(name, kind, m, n, k, act="silu", train=False):
        return dict(name=name, op="gated", kind=kind, m=m, n=n, k=k, act=act, bias=False, residual=False, train=train)

    return [
        # attention's output projection for one token of one request, added to the residual stream
        fused("fused fp8 1 token", "e4m3", 1, 4096, 4096, "none", False, True),
        # the down projection for a batch of single tokens, an odd number of them
        fused("fused fp8 37 tokens", "e4m3", 37, 4096, 14336, "none", False, True),
        # the down projection of a prompt, added to the residual stream
        fused("fused fp8 prompt", "e4m3", 2048, 4096, 14336, "none", False, True),
        # an ungated block's first projection with bias and activation, ragged sizes, E5M2 tokens
        fused("fused fp8 ragged", "mixed", 777, 1003, 2064, "gelu", True, False),
        # a training step of a projection with bias, activation and residual
        fused("fused bf16 train", "bf16", 2048, 4096, 4096, "gelu_tanh", True, True, True),
        # the same on ragged sizes
        fused("fused bf16 train ragged", "bf16", 301, 1111, 520, "silu", True, True, True),
        # gate and up projections for one token
        gated("gated fp8 1 token", "e4m3", 1, 14336, 4096),
        # and for a full decode batch
        gated("gated fp8 64 tokens", "e4m3", 64, 14336, 4096),
        # a long prompt
        gated("gated fp8 prompt", "e4m3", 8192, 14336, 4096),
        # BF16 weights, a few tokens, a narrow block
        gated("gated bf16 16 tokens", "bf16", 16, 4096, 2048, "gelu"),
        # a training step of a transformer's feed-forward block
        gated("gated bf16 train", "bf16", 4096, 14336, 4096, "silu", True),
        # the same on ragged sizes
        gated("gated bf16 train ragged", "bf16", 1000, 1365, 1000, "gelu_tanh", True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("fused", "gated"))
    kind = rng.choice(("e4m3", "e4m3", "e5m2", "mixed", "bf16", "bf16", "bf16", "bf16"))
    train = kind == "bf16" and rng.random() < 0.6
    grain = 8 if kind == "bf16" else 16
    while True:
        m = spread(1, 8192)
        n = spread(24, 14336)
        k = max(grain, spread(64, 14336) // grain * grain)
        products = (2 if op == "gated" else 1) * (3 if train else 1)
        if products * m * n * k <= 6 * 4096 * 14336 * 4096:
            break
    fused = op == "fused"
    return dict(op=op, kind=kind, m=m, n=n, k=k, act=rng.choice(ACTS if fused else ACTS[1:]),
                bias=fused and rng.random() < 0.5, residual=fused and rng.random() < 0.5, train=train)


def _types(kind):
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    return {"e4m3": (e4, e4), "e5m2": (e5, e5), "mixed": (e5, e4), "bf16": (torch.bfloat16, torch.bfloat16)}[kind]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    m, n, k = case["m"], case["n"], case["k"]
    ta, tb = _types(case["kind"])

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std)

    def tokens():
        """Activations N(0, 1), and for FP8 the scale of each row that takes its largest value to 256."""
        x = normal(m, k)
        if case["kind"] == "bf16":
            return x.to(ta), None
        s = x.abs().amax(dim=1).clamp_(min=1e-6) / 256.0
        return (x / s[:, None]).to(ta), s

    def weights():
        """Weights N(0, 0.02^2), and for FP8 the scale of each channel that takes its largest value to 448."""
        w = normal(n, k, std=0.02)
        if case["kind"] == "bf16":
            return w.to(tb), None
        s = w.abs().amax(dim=1).clamp_(min=1e-6) / 448.0
        return (w / s[:, None]).to(tb), s

    s = dict(case)
    s["a"], s["sa"] = tokens()
    if case["op"] == "fused":
        s["b"], s["sb"] = weights()
        s["bias_v"] = normal(n, std=0.5) if case["bias"] else None
        s["res"] = normal(m, n).bfloat16() if case["residual"] else None
    else:
        s["wg"], s["sg"] = weights()
        s["wu"], s["su"] = weights()
    if case["train"]:
        s["grad"] = normal(m, n).bfloat16()
    return s


# ---------------------------------------------------------------------------
# The plain form: 32-bit products and elementary operations.
# ---------------------------------------------------------------------------
def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
    return z / (1 + torch.exp(-2 * u))


def _act_slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    u = c * (z + 0.044715 * z * z * z)
    s = 1 / (1 + torch.exp(-2 * u))
    return s + z * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * z * z)


def _product(a, b, sa, sb):
    z = a.float() @ b.float().t()
    if sa is not None:
        z = z * (sa[:, None] * sb[None, :])
    return z


def _plain(s):
    bf = torch.bfloat16
    if s["op"] == "fused":
        z = _product(s["a"], s["b"], s["sa"], s["sb"])
        if s["bias_v"] is not None:
            z = z + s["bias_v"]
        d = _act(s["act"], z)
        if s["res"] is not None:
            d = d + s["res"].float()
        out = {"d": d.to(bf)}
        if s["train"]:
            dz = s["grad"].float() * _act_slope(s["act"], z)
            out["grad_a"] = (dz @ s["b"].float()).to(bf)
            out["grad_b"] = (dz.t() @ s["a"].float()).to(bf)
            if s["bias_v"] is not None:
                out["grad_bias"] = dz.sum(dim=0, dtype=torch.float64).float()
        return out
    gate = _product(s["a"], s["wg"], s["sa"], s["sg"])
    up = _product(s["a"], s["wu"], s["sa"], s["su"])
    act = _act(s["act"], gate)
    out = {"h": (act * up).to(bf)}
    if s["train"]:
        dh, a = s["grad"].float(), s["a"].float()
        dg = dh * up * _act_slope(s["act"], gate)
        du = dh * act
        out["grad_a"] = (dg @ s["wg"].float() + du @ s["wu"].float()).to(bf)
        out["grad_gate"] = (dg.t() @ a).to(bf)
        out["grad_up"] = (du.t() @ a).to(bf)
    return out


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp8_gemm_amd as f

    fp8 = s["kind"] != "bf16"
    if s["op"] == "fused":
        if fp8:
            return {"d": f.gemm_nt_fused(s["a"], s["b"], s["sa"], s["sb"], bias=s["bias_v"], activation=s["act"],
                                         residual=s["res"])}
        if not s["train"]:
            return {"d": f.gemm_nt_bf16_fused(s["a"], s["b"], bias=s["bias_v"], activation=s["act"],
                                              residual=s["res"])}
        pre = None
        if s["act"] != "none":
            pre = torch.empty((s["m"], s["n"]), dtype=torch.float32, device=s["a"].device)
        d = f.gemm_nt_bf16_fused(s["a"], s["b"], bias=s["bias_v"], activation=s["act"], residual=s["res"], preact=pre)
        ga, gb, gbias = f.gemm_nt_bf16_fused_backward(s["grad"], s["a"], s["b"], activation=s["act"], preact=pre,
                                                      bias_grad=s["bias_v"] is not None)
        out = {"d": d, "grad_a": ga, "grad_b": gb}
        if s["bias_v"] is not None:
            out["grad_bias"] = gbias
        return out
    if fp8:
        return {"h": f.gated_nt(s["a"], s["wg"], s["wu"], s["sa"], s["sg"], s["su"], activation=s["act"])}
    if not s["train"]:
        return {"h": f.gated_nt_bf16(s["a"], s["wg"], s["wu"], activation=s["act"])}
    pre = torch.empty((2, s["m"], s["n"]), dtype=torch.float32, device=s["a"].device)
    h = f.gated_nt_bf16(s["a"], s["wg"], s["wu"], activation=s["act"], preact=pre)
    ga, gg, gu = f.gated_nt_bf16_backward(s["grad"], s["a"], s["wg"], s["wu"], pre, activation=s["act"])
    return {"h": h, "grad_a": ga, "grad_gate": gg, "grad_up": gu}


def work(case):
    m, n, k = case["m"], case["n"], case["k"]
    e = 2 if case["kind"] == "bf16" else 1
    w = 2 if case["op"] == "gated" else 1
    nbytes = e * (m * k + w * n * k) + 2 * m * n            # tokens, weights, output
    if e == 1:
        nbytes += 4 * (m + w * n)                           # scales
    nbytes += (4 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
    flops = 2 * w * m * n * k
    if case["train"]:
        # the output's gradient in, those of the tokens, the weights and the bias out; two more products of each kind
        nbytes += 2 * m * n + 2 * (m * k + w * n * k) + (4 * n if case["bias"] else 0)
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# The definition in 64 bits.
# ---------------------------------------------------------------------------
def _act64(name, z):
    """(act(z), act'(z)) in float64."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        v, dv = z, torch.ones_like(z)
    else:
        c = math.sqrt(8 / math.pi)
        v, dv = c * (z + 0.044715 * z ** 3), c * (1 + 0.134145 * z ** 2)
    s = torch.special.expit(v)
    return z * s, s + z * s * torch.special.expit(-v) * dv


def exact(case, seed):
    s = prepare(case, seed)
    a = s["a"].double()
    one = torch.ones((), dtype=torch.float64, device=a.device)
    sa = one if s["sa"] is None else s["sa"].double().unsqueeze(1)

    def preact(w, sw):
        z = torch.mm(a, w.double().t())
        return z * sa * (one if sw is None else sw.double().unsqueeze(0))

    if s["op"] == "fused":
        z = preact(s["b"], s["sb"])
        if s["bias_v"] is not None:
            z += s["bias_v"].double()
        v, dv = _act64(s["act"], z)
        out = {"d": v if s["res"] is None else v + s["res"].double()}
        if s["train"]:
            dz = s["grad"].double() * dv
            out["grad_a"] = torch.mm(dz, s["b"].double())
            out["grad_b"] = torch.mm(dz.t(), a)
            if s["bias_v"] is not None:
                out["grad_bias"] = dz.sum(dim=0)
        return out
    gate, up = preact(s["wg"], s["sg"]), preact(s["wu"], s["su"])
    v, dv = _act64(s["act"], gate)
    out = {"h": v * up}
    if s["train"]:
        dh = s["grad"].double()
        dg = dh * up * dv
        du = dh * v
        out["grad_a"] = torch.mm(dg, s["wg"].double()) + torch.mm(du, s["wu"].double())
        out["grad_gate"] = torch.mm(dg.t(), a)
        out["grad_up"] = torch.mm(du.t(), a)
    return out
