"""Operands and outputs of the fused products within one buffer."""
import pytest
import torch

from tests.test_gpu_fused import BF, DEV, E4, f, rand  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [5, 70, 2100])
def test_columns_of_one_buffer(f, M):
    N, K = 136, 64
    x, w, res = rand(1, M, K), rand(2, N, K), rand(3, M, N)
    want = f.gemm_nt_bf16_fused(x, w, activation="gelu", residual=res)
    buf = torch.full((M, K + 2 * N), 7.0, dtype=BF, device=DEV)
    a, r, out = buf[:, :K], buf[:, K:K + N], buf[:, K + N:]
    a.copy_(x)
    r.copy_(res)
    assert f.gemm_nt_bf16_fused(a, w, activation="gelu", residual=r, out=out) is out
    assert torch.equal(out, want) and torch.equal(a, x) and torch.equal(r, res)
    # pre-activations in rows between each other's
    pre = torch.empty(M, 2, N, device=DEV).transpose(0, 1)
    two = torch.empty(2, M, N, device=DEV)
    assert torch.equal(f.gated_nt_bf16(x, w, w.flip(0).contiguous(), preact=pre),
                       f.gated_nt_bf16(x, w, w.flip(0).contiguous(), preact=two)) and torch.equal(pre, two)


@pytest.mark.parametrize("M", [5, 70, 2100])
def test_overlaps_are_refused(f, M):
    N, K = 64, 64
    a8, b8 = rand(1, M, K, dtype=E4), rand(2, N, K, dtype=E4)
    x, w = rand(3, M, K), rand(4, N, K)
    buf = torch.full((M + 1, N + 8), 7.0, dtype=BF, device=DEV)
    before, pre = buf.clone(), torch.zeros(2 * M, N, device=DEV)
    for call in (lambda: f.gemm_nt_fused(a8, b8, residual=buf[1:, :N], out=buf[:M, :N]),
                 lambda: f.gemm_nt_bf16_fused(x, w, residual=buf[:M, 8:], out=buf[:M, :N]),
                 lambda: f.gemm_nt_bf16_fused(buf[:M, :K], w, out=buf[:M, :N]),
                 lambda: f.gemm_nt_bf16_fused(x, w, out=pre.view(BF)[:M, :N], preact=pre[:M]),
                 lambda: f.gated_nt_bf16(x, w, w, preact=torch.as_strided(pre, (2, M, N), (N // 2, 2 * N, 1)))):
        with pytest.raises((f.Fp8GemmError, ValueError), match="overlap"):
            call()
    torch.cuda.synchronize()
    assert torch.equal(buf, before) and not pre.any()
