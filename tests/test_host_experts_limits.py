"""Sizes at the experts' and integer entry points' limits, and shapes that hold as many elements in another order (CPU
only: fake addresses, no kernel launch)."""
import pytest
import torch

from tests.test_host_experts import CALLS
from tests.test_host_fused import call, f  # noqa: F401 (f: fixture)
from tests.test_host_fused_overlap import UNSUPPORTED, at, without_gpu

FAR = dict(X=at(0), Q=at(0) + (1 << 45), s=at(0) + (1 << 46))


@without_gpu
@pytest.mark.parametrize("M,K", [((1 << 24) - 1, 64), (1 << 24, 64), (1 << 26, 1024), ((1 << 31) - 1, 16), ((1 << 31) - 1, 2048),
                                 (1 << 22, 8208), (1 << 24, 14336), (1 << 22, 70000)])
def test_quantise_takes_any_number_of_rows(f, M, K):  # noqa: F811
    st, msg = call(f, "int8_quantize_rows", *CALLS["int8_quantize_rows"], M=M, K=K, ldx=K, ldq=K, **FAR)
    assert st == UNSUPPORTED, msg


def test_transposed_channel_scales_are_refused(f):  # noqa: F811
    a, o = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(3, dtype=torch.int32)
    for N, shape in ((8, (8, 2)), (8, (8, 2, 1)), (16, (16, 2))):
        with pytest.raises(ValueError, match="scale_b must be"):
            f.grouped_gemm_ragged_int8(a, torch.zeros(2, N, 32, dtype=torch.int8), o, scale_b=torch.ones(shape))
    # the same order in another shape goes on (to the check of the device)
    for shape in ((2, 8), (16,), (16, 1), (2, 8, 1), (1, 16)):
        with pytest.raises(ValueError, match="GPU"):
            f.grouped_gemm_ragged_int8(a, torch.zeros(2, 8, 32, dtype=torch.int8), o, scale_b=torch.ones(shape))
    with pytest.raises(ValueError, match="GPU"):
        f.grouped_gemm_ragged_int8(a, torch.zeros(1, 8, 32, dtype=torch.int8), o[:2], scale_b=torch.ones(8, 1))


@pytest.mark.parametrize("m,n", [((1 << 31) - 1, 5), (1, (1 << 30) + 8), (64, (1 << 30) + 8), (1, (1 << 31) - 1)])
def test_chosen_classes_fit_a_launch(f, m, n):  # noqa: F811
    """A launch holds fewer than 2^32 threads along a dimension of its grid (the largest outputs that memory holds)."""
    for p in (f.experts_plan(4, m, n, 16), f.fused_plan(0, m, n, 16), f.fused_plan(2, m, n, 16)):
        assert p.workgroups // (-(-m // 64) if p.variant == 4 else 1) < 1 << 24, (p.variant, p.workgroups)


@pytest.mark.parametrize("op,m,n,k,g,runs", [
    (1, 64, 64, 131056, 4, True), (1, 64, 64, 131072, 4, False), (4, 64, 64, 131056, 1, True), (4, 64, 64, 131072, 1, False),
    (4, 3000, 5000, 131072, 1, False), (0, 64, 64, 131072, 4, True), (2, 1 << 30, 64, 64, 4, True), (2, (1 << 30) + 1, 64, 64, 4, False),
    (3, 1 << 30, 64, 64, 4, True), (3, (1 << 30) + 1, 64, 64, 4, False), (3, 64, 4194296, 1 << 20, 8, True),
    (3, 64, 4194296, 1 << 20, 65535, False), (0, (1 << 31) - 1, 4194296, 64, 4, False),
])
def test_plan_of_refused_sizes_names_no_kernel(f, op, m, n, k, g, runs):  # noqa: F811
    p = f.experts_plan(op, m, n, k, g)
    assert (p.variant != 0) == runs == (p.workgroups != 0)
