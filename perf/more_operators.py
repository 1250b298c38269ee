"""Experts' products over ragged groups of rows and products in 8-bit integers, as they are measured.

Four operators.  An expert layer sorts its token rows by expert: the rows offsets[g] .. offsets[g + 1] - 1 belong to
expert g, any number of them, and rows behind offsets[G] (a padded batch) to none.

  experts    (BF16)  D[r] = A[r] . B[g]^T for the rows r of expert g; the rows of none stay as they were
             backward: dA[r] = dD[r] . B[g] (0 for the rows of none),  dB[g] = sum over g's rows of dD[r]^T . A[r]
  int8       D = act(sa[m] sb[n] (A . B^T) + bias[n]) + R, A and B in 8-bit integers, a scale for each token and each
             channel; `dynamic`: A is quantised from BF16 first
  experts8   (8-bit integers)  D[r] = sa[r] sb[g] (A[r] . B[g]^T)
  quantise   sa[m] = max_k |X[m, k]| / 127,  A[m, k] = the whole number nearest to X[m, k] / sa[m], ties to even; a row
             of zeros has the scale 0

A is [M, K] (token rows), B [N, K] or [G, N, K] (weights), all K-contiguous.  A case names its operator (`op`) and its
sizes; `tokens` tokens with `topk` different experts each make the rows of the experts' operators, `tail` rows of no
expert follow them.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    def experts(name, op, tokens, topk, g, n, k, tail=0, train=False):
        return dict(name=name, op=op, tokens=tokens, topk=topk, g=g, n=n, k=k, tail=tail, train=train)

    def int8(name, m, n, k, act="none", bias=False, residual=False, dynamic=False):
        return dict(name=name, op="int8", m=m, n=n, k=k, act=act, bias=bias, residual=residual, dynamic=dynamic)

    return [
        # one token of one request through its 8 experts' first projection
        experts("experts bf16 1 token", "experts", 1, 8, 64, 2048, 4096),
        # a decode batch padded to a captured size: a few rows for each of 64 experts
        experts("experts bf16 decode", "experts", 64, 8, 64, 2048, 4096, tail=128),
        # a training step of a layer of few wide experts: product and both gradients
        experts("experts bf16 train", "experts", 4096, 2, 8, 14336, 4096, train=True),
        # the same with many narrow experts and odd sizes, of which some may see no row
        experts("experts bf16 train ragged", "experts", 1111, 3, 17, 1032, 2056, tail=45, train=True),
        # attention's output projection for one token, quantised in the same call, added to the residual stream
        int8("int8 1 token", 1, 4096, 4096, residual=True, dynamic=True),
        # a feed-forward block's first projection for a full decode batch
        int8("int8 64 tokens", 64, 14336, 4096),
        # the same for a prompt
        int8("int8 prompt", 4096, 14336, 4096),
        # odd sizes, bias and activation
        int8("int8 ragged", 777, 1003, 2064, "gelu", bias=True),
        # experts with 8-bit weights: a decode batch
        experts("experts int8 decode", "experts8", 64, 8, 64, 2048, 7168),
        # and a long prompt
        experts("experts int8 prompt", "experts8", 8192, 8, 64, 2048, 4096, tail=77),
        # the inputs of a down projection for a small batch of single tokens
        dict(name="quantise 16 tokens", op="quantise", m=16, k=14336),
        # and for a prompt
        dict(name="quantise prompt", op="quantise", m=8192, k=14336),
    ]


def draw(rng):
    def spread(lo, hi, grain=1):
        return max(grain, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) // grain * grain)

    op = rng.choice(("experts", "experts", "int8", "experts8", "quantise"))
    if op == "quantise":
        while True:
            m, k = spread(1, 16384), spread(16, 32768, 16)
            if m * k <= 8192 * 14336:
                return dict(op=op, m=m, k=k)
    most = 3 * 8192 * 14336 * 4096
    if op == "int8":
        while True:
            m, n, k = spread(1, 8192), spread(24, 28672), spread(64, 28672, 16)
            if m * n * k <= most and n * k <= 2e8:
                break
        dynamic = rng.random() < 0.5
        return dict(op=op, m=m, n=n, k=k, act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    dynamic=dynamic)
    train = op == "experts" and rng.random() < 0.6
    while True:
        g = spread(2, 160)
        topk = rng.randint(1, min(8, g))
        tokens = spread(1, 8192)
        n, k = spread(32, 14336, 8), spread(64, 8192, 8 if op == "experts" else 16)
        if (3 if train else 1) * tokens * topk * n * k <= most and g * n * k <= 5e8:
            break
    tail = rng.choice((0, 0, 1, 100, spread(1, 512)))
    return dict(op=op, tokens=tokens, topk=topk, g=g, n=n, k=k, tail=tail, train=train)


def _rows(case):
    return case["tokens"] * case["topk"] + case["tail"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, k = case["op"], case["k"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std)

    def activations(m):
        """N(0, 1) with one channel in 64 ten times as large, as a transformer's residual stream has them; in batches
        the last row is a padding token's, zeros."""
        x = normal(m, k)
        x[:, ::64] *= 10.0
        if m > 2:
            x[-1].zero_()
        return x.bfloat16()

    def codes(x):
        """Rows of x in 8-bit integers, and their scales."""
        scale = x.abs().amax(dim=-1).clamp_(min=1e-12) / 127.0
        return torch.round(x / scale.unsqueeze(-1)).to(torch.int8), scale

    s = dict(case)
    if op == "quantise":
        s["x"] = activations(case["m"])
        return s
    n = case["n"]
    if op == "int8":
        m = case["m"]
        if case["dynamic"]:
            s["x"] = activations(m)
        else:
            s["a"], s["sa"] = codes(normal(m, k))
        s["b"], s["sb"] = codes(normal(n, k, std=0.02))
        s["bias_v"] = normal(n, std=0.5) if case["bias"] else None
        s["res"] = normal(m, n).bfloat16() if case["residual"] else None
        return s
    # the experts that each token is sent to, some more popular than others; the rows sorted by expert
    g, m = case["g"], _rows(case)
    popular = torch.exp(normal(g, std=0.5)).expand(case["tokens"], g)
    chosen = torch.multinomial(popular, case["topk"], replacement=False, generator=gen)
    counts = torch.bincount(chosen.reshape(-1), minlength=g)
    s["offsets"] = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
    s["most"] = int(counts.max())                          # (the plain form pads every expert's rows to this)
    x, w = normal(m, k), normal(g, n, k, std=0.02)
    if op == "experts":
        s["a"], s["b"] = x.bfloat16(), w.bfloat16()
        if case["train"]:
            s["grad"] = normal(m, n).bfloat16()
    else:
        s["a"], s["sa"] = codes(x)
        s["b"], s["sb"] = codes(w)
    # a captured step's output buffer, whose rows behind the last expert nothing writes
    s["out"] = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda") if case["tail"] else None
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


def _quantise(x):
    """Codes and scales of the rows of x: the quotient in 64 bits, next to whose halves a rounding would show."""
    most = x.double().abs().amax(dim=1, keepdim=True)
    codes = torch.round(x.double() * 127 / torch.where(most > 0, most, torch.ones_like(most)))
    return codes.to(torch.int8), (most[:, 0] / 127).float()


def _padded_rows(s):
    """[G, most] row numbers, those past an expert's last row being M (an extra row of zeros)."""
    at = torch.arange(s["most"], device=s["a"].device)
    first, last = s["offsets"][:-1, None], s["offsets"][1:, None]
    return torch.where(first + at < last, first + at, s["a"].shape[0])


def _with_zero_row(t):
    return torch.cat((t.float(), torch.zeros(1, t.shape[1], device=t.device)))


def _scatter(rows, y, m):
    """The rows of y [G, most, C] at their places among m; zeros where no expert has a row."""
    out = torch.zeros(m + 1, y.shape[2], device=y.device)
    out[rows.reshape(-1)] = y.reshape(-1, y.shape[2])
    return out[:m]


def _plain_experts(s):
    rows, m = _padded_rows(s), s["a"].shape[0]
    a, b = _with_zero_row(s["a"])[rows], s["b"].float()
    y = torch.bmm(a, b.transpose(1, 2))
    if s["op"] == "experts8":
        sa = _with_zero_row(s["sa"][:, None])[rows]
        y = y * (sa * s["sb"][:, None, :])
    out = {"d": _scatter(rows, y, m).to(torch.bfloat16)}
    if s["train"]:
        g = _with_zero_row(s["grad"])[rows]
        out["grad_a"] = _scatter(rows, torch.bmm(g, b), m).to(torch.bfloat16)
        out["grad_b"] = torch.bmm(g.transpose(1, 2), a).to(torch.bfloat16)
    return out


def _plain(s):
    if s["op"] == "quantise":
        codes, scales = _quantise(s["x"])
        return {"codes": codes, "scales": scales}
    if s["op"] != "int8":
        return _plain_experts(s)
    a, sa = _quantise(s["x"]) if s["dynamic"] else (s["a"], s["sa"])
    z = a.float() @ s["b"].float().t() * (sa[:, None] * s["sb"][None, :])
    if s["bias_v"] is not None:
        z = z + s["bias_v"]
    d = _act(s["act"], z)
    if s["res"] is not None:
        d = d + s["res"].float()
    return {"d": d.to(torch.bfloat16)}


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp8_gemm_amd as f

    if s["op"] == "quantise":
        codes, scales = f.quantize_rows_int8(s["x"])
        return {"codes": codes, "scales": scales}
    if s["op"] == "int8":
        a, sa = f.quantize_rows_int8(s["x"]) if s["dynamic"] else (s["a"], s["sa"])
        return {"d": f.gemm_nt_int8(a, s["b"], sa, s["sb"], bias=s["bias_v"], activation=s["act"], residual=s["res"])}
    if s["op"] == "experts8":
        return {"d": f.grouped_gemm_ragged_int8(s["a"], s["b"], s["offsets"], s["sa"], s["sb"], out=s["out"])}
    out = {"d": f.grouped_gemm_ragged_bf16(s["a"], s["b"], s["offsets"], out=s["out"])}
    if s["train"]:
        out["grad_a"], out["grad_b"] = f.grouped_gemm_ragged_bf16_backward(s["grad"], s["a"], s["b"], s["offsets"])
    return out


def work(case):
    k = case["k"]
    if case["op"] == "quantise":
        m = case["m"]
        return {"bytes": 3 * m * k + 4 * m, "flops": 2 * m * k}
    n = case["n"]
    if case["op"] == "int8":
        m = case["m"]
        nbytes = (2 if case["dynamic"] else 1) * m * k + n * k + 2 * m * n + 4 * n + (0 if case["dynamic"] else 4 * m)
        nbytes += (4 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
        return {"bytes": nbytes, "flops": 2 * m * n * k}
    m, g = case["tokens"] * case["topk"], case["g"]
    # the experts that have a row, at the mean of as many draws (a little high: some experts are more popular)
    seen = g * (1 - (1 - case["topk"] / g) ** case["tokens"])
    e = 2 if case["op"] == "experts" else 1
    nbytes = e * (m * k + seen * n * k) + 2 * m * n + 4 * (g + 1)
    if e == 1:
        nbytes += 4 * (m + seen * n)
    flops = 2 * m * n * k
    if case["train"]:
        # the output's gradient in, those of the rows and of every expert's weights out; two more products
        nbytes += 2 * m * n + 2 * ((m + case["tail"]) * k + g * n * k)
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# The definition in 64 bits.
# ---------------------------------------------------------------------------
def _act64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    v = z if name == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.special.expit(v)


def _quantise64(x):
    """(codes, scales): n = floor(q + 1/2), less 1 where q + 1/2 is an odd whole number n (a tie)."""
    x = x.double()
    most = x.abs().max(dim=1).values
    q = 127 * x / most.clamp(min=1e-300).unsqueeze(1)
    n = torch.floor(q + 0.5)
    odd = torch.remainder(n, 2) == 1
    n -= (odd & (q + 0.5 == n)).double()
    return n.to(torch.int8), most / 127


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        codes, scales = _quantise64(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "int8":
        if case["dynamic"]:
            s["a"], sa = _quantise64(s["x"])
        else:
            sa = s["sa"].double()
        z = torch.mm(s["a"].double(), s["b"].double().t())
        z *= sa.unsqueeze(1)
        z *= s["sb"].double().unsqueeze(0)
        if s["bias_v"] is not None:
            z += s["bias_v"].double()
        d = _act64(case["act"], z)
        return {"d": d if s["res"] is None else d + s["res"].double()}
    bounds = s["offsets"].tolist()
    m, n, k = s["a"].shape[0], case["n"], case["k"]
    out = {"d": torch.zeros(m, n, dtype=torch.float64, device="cuda")}
    if case["train"]:
        out["grad_a"] = torch.zeros(m, k, dtype=torch.float64, device="cuda")
        out["grad_b"] = torch.zeros(case["g"], n, k, dtype=torch.float64, device="cuda")
    for e in range(case["g"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        a, b = s["a"][lo:hi].double(), s["b"][e].double()
        y = torch.mm(a, b.t())
        if op == "experts8":
            y = y * s["sa"][lo:hi].double().unsqueeze(1) * s["sb"][e].double().unsqueeze(0)
        out["d"][lo:hi] = y
        if case["train"]:
            g = s["grad"][lo:hi].double()
            out["grad_a"][lo:hi] = torch.mm(g, b)
            out["grad_b"][e] = torch.mm(g.t(), a)
    return out
