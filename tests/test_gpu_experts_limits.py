"""The ragged product at the largest number of rows that it accepts."""
import pytest
import torch

from tests import _experts as E
from tests import _fused as F
from tests._experts import BF, DEV, rand
from tests.test_gpu_experts import f  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("end", [(1 << 31) - 1, (1 << 31) - 256])
def test_most_rows(f, end):  # noqa: F811
    """One expert with 2^31 - 1 rows, whose number of tiles is counted past 2^31, and with the most that is not; rows of
    zeros but for some, all of which are written."""
    M, N, K = (1 << 31) - 1, 8, 8
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("takes 69 GB and temporaries")
    assert f.experts_plan(0, M, N, K, 2).tile_m == 256     # (the class that this number of rows takes)
    rows = torch.tensor([0, 255, 256, 1 << 20, (1 << 30) + 3, end - 300, end - 257, end - 256, end - 1], device=DEV)
    a = torch.zeros(M, K, dtype=BF, device=DEV)
    a[rows] = rand(1, len(rows), K)
    b = rand(2, 2, N, K)
    out = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    offsets = torch.tensor([0, end, end], dtype=torch.int64).to(torch.int32).to(DEV)
    f.grouped_gemm_ragged_bf16(a, b, offsets, out=out)
    z, S, hw = F.product(a[rows], b[0])
    F.check(out[rows], z, 1e-5 * S, hw, K, "most rows")
    assert (out[end:] == 7).all()
    out[rows] = 0
    assert not any(bool(part.any()) for part in out[:end].split(1 << 27))
