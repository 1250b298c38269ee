"""The plan of the gated form's weight gradients, two products in one launch,
and the workspaces that follow from the plans (CPU only)."""
import pytest

from tests.test_host_fused import f  # noqa: F401 (fixture)

SHAPES = [(0, 0, 0), (1, 1, 8), (64, 64, 64), (65, 129, 1000), (5, 14336, 4096), (8192, 128, 128), (4000, 36, 3000),
          (9000, 130, 520), (12000, 1030, 1032), (4096, 14336, 4096)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_workspaces_hold_the_split_sums(f, M, N, K):  # noqa: F811
    lib = f.load_library()
    cols = (N + 63) // 64 * 64

    def sums(op, m, n, k):
        splits = f.fused_plan(op, m, n, k).k_splits if K else 1
        return 0 if splits == 1 else 4 * splits * m * n * (2 if op > 4 else 1)

    need = 4 * M * cols + max(sums(4, M, K, 2 * cols), sums(4 + f.PLAN_PAIR, N, K, M))
    assert need <= lib.bf16_gated_nt_backward_workspace(M, N, K) < need + 256
    # (the bias gradient's partial sums: a float per column and block of 8 to 64 rows)
    need = 2 * M * cols + max(sums(4, M, K, cols), sums(4, N, K, M))
    assert need + 4 * N * (-(-M // 64)) <= lib.bf16_gemm_nt_fused_backward_workspace(M, N, K) < need + 512 + 4 * N * (-(-M // 8))


@pytest.mark.parametrize("n,k,m", [(36, 3000, 4000), (130, 520, 9000), (1030, 1032, 12000), (14336, 4096, 4096), (64, 64, 64)])
def test_pair_plan(f, n, k, m):  # noqa: F811
    pair, one = f.fused_plan(4 + f.PLAN_PAIR, n, k, m), f.fused_plan(4, n, k, m)
    tiles = -(-n // pair.tile_m) * -(-k // pair.tile_n)
    assert pair.workgroups == 2 * tiles * pair.k_splits
    # two products fill the device with fewer splits of each
    assert 1 <= pair.k_splits <= 64 and 2 * 4 * pair.k_splits * n * k * (pair.k_splits > 1) <= 128 << 20
    if (pair.tile_m, pair.tile_n) == (one.tile_m, one.tile_n):
        assert pair.k_splits <= one.k_splits


def test_pair_splits_less_than_one(f):  # noqa: F811
    assert f.fused_plan(4 + f.PLAN_PAIR, 36, 3000, 4000).k_splits < f.fused_plan(4, 36, 3000, 4000).k_splits


@pytest.mark.parametrize("op", [0, 1, 2, 3, 5])
def test_pair_is_of_backward_products(f, op):  # noqa: F811
    with pytest.raises(f.Fp8GemmError) as e:
        f.fused_plan(op + f.PLAN_PAIR, 64, 64, 64)
    assert e.value.status == -8
