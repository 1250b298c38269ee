"""Experts' and integer products of as many tiles and workgroups as memory allows: more than 2^24 of them, which the
64-bit sizes of thin matrices reach."""
import pytest
import torch

from tests import _fused as F
from tests._experts import BF, DEV, codes, rand
from tests.test_gpu_experts import f  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def needs(gb):
    if torch.cuda.mem_get_info()[0] < (gb + 16) << 30:
        pytest.skip(f"takes {gb} GB and temporaries")


def offsets(*ends):
    return torch.tensor(ends, dtype=torch.int64).to(torch.int32).to(DEV)


def zero(t):
    return not any(bool(part.any()) for part in t.split(max(1, (1 << 30) // t[0].numel())))


@pytest.mark.parametrize("N", [5, 8])
def test_most_rows_of_integers(f, N):  # noqa: F811
    """Dense (staged and direct epilogue) and ragged, 2^31 - 1 rows of 16 codes."""
    M, K = (1 << 31) - 1, 16
    needs(72)
    rows = torch.tensor([0, 127, 128, 255, 256, 1 << 20, (1 << 30) + 3, M - 256, M - 128, M - 1], device=DEV)
    a = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    a[rows] = codes(1, len(rows), K)
    b = codes(2, N, K)
    want = (a[rows].float() @ b.float().t()).to(BF)
    out = torch.full((M, 8), 7.0, dtype=BF, device=DEV)
    for ragged in (False, True):
        if ragged and N % 8:
            continue
        if ragged:
            f.grouped_gemm_ragged_int8(a, b[None], offsets(0, M), out=out)
        else:
            f.gemm_nt_int8(a, b, out=out[:, :N])
        assert torch.equal(out[rows, :N], want)
        out[rows, :N] = 0
        assert zero(out[:, :N]) and (N == 8 or all(bool((part == 7).all()) for part in out[:, N:].split(1 << 28)))
        out.fill_(7.0)


@pytest.mark.parametrize("M", [1, 3])
def test_most_columns_of_integers(f, M):  # noqa: F811
    """2^30 and some channels: more workgroups of the few-token kernel than a launch holds."""
    N, K = (1 << 30) + 8, 16
    needs(20 + 3 * M)
    assert f.experts_plan(4, M, N, K).workgroups < 1 << 24
    a = codes(1, M, K)
    g = torch.Generator(device=DEV).manual_seed(2)
    b = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8, device=DEV)
    out = f.gemm_nt_int8(a, b)
    for at in range(0, N, 1 << 26):
        part = b[at:at + (1 << 26)].float()
        want = sum(a[:, k:k + 1].float() * part[:, k] for k in range(K)).to(BF)       # (exact: sums below 2^24)
        assert torch.equal(out[:, at:at + (1 << 26)], want)


def test_many_experts_few_rows(f):  # noqa: F811
    """2^24 workgroups of the few-token kernel: 4096 experts of 2^20 channels."""
    M, G, N, K = 1024, 4096, 1 << 20, 16
    needs(74)
    assert f.experts_plan(1, M, N, K, G).variant == 4 and f.experts_plan(1, M, N, K, G).workgroups >= 1 << 24
    b = torch.zeros(G, N, K, dtype=torch.int8, device=DEV)
    b[5], b[4095] = codes(1, N, K), codes(2, N, K)
    a = codes(3, M, K)
    out = f.grouped_gemm_ragged_int8(a, b, offsets(*[0] * 6, *[1000] * (G - 6), M))
    for lo, hi, g in ((0, 1000, 5), (1000, M, 4095)):
        for at in range(0, N, 1 << 17):
            cols = slice(at, at + (1 << 17))
            want = sum(a[lo:hi, k:k + 1].float() * b[g, cols, k].float() for k in range(K)).to(BF)
            assert torch.equal(out[lo:hi, cols], want)


def test_many_weight_gradients(f):  # noqa: F811
    """2^25 tiles of weight gradients: 65535 experts of 65536 x 16, of which three have rows."""
    M, G, N, K = 1024, 65535, 65536, 16
    needs(140)
    assert f.experts_plan(3, M, N, K, G).workgroups > 1 << 24
    grad, a = rand(1, M, N), rand(2, M, K)
    b = torch.zeros(K, dtype=BF, device=DEV).expand(G, N, K)   # (not read: the weight gradients alone)
    o = offsets(0, *[300] * 7, *[310] * (G - 8), M)
    _, gb = f.grouped_gemm_ragged_bf16_backward(grad, a, b, o, a_grad=False)
    cols = torch.cat((torch.arange(0, 300), torch.arange(N - 300, N)))
    for g, lo, hi in ((0, 0, 300), (7, 300, 310), (G - 1, 310, M)):
        g6 = grad[lo:hi].cpu().double()[:, cols].t()
        F.check(gb[g][cols.to(DEV)], *F.backward_products(g6, torch.zeros_like(g6), a[lo:hi]), hi - lo, f"expert {g}")
        gb[g].zero_()
    assert zero(gb)
