"""Sizes at the experts' and integer entry points' limits (CPU only: fake addresses, no kernel launch)."""
import pytest

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
