"""The quantisation of more rows than one launch holds, against 64-bit references (tests/_experts.py)."""
import pytest
import torch

from tests import _experts as E
from tests._experts import BF, DEV, rand
from tests.test_gpu_experts import f  # noqa: F401 (f: fixture)

pytestmark = pytest.mark.gpu


def check_rows(x, q, s, rows):
    want, scale = E.quantised(x[rows])
    assert torch.equal(q[rows].cpu(), want)
    assert ((s[rows].cpu().double() - scale).abs() <= 2.0 ** -24 * scale + 2.0 ** -150).all()


def test_many_short_rows(f):  # noqa: F811
    """2^26 and some rows of 16 values, four to a workgroup: the second launch begins at row 2^26 - 4."""
    first, K = 4 * (2 ** 24 - 1), 16
    M = first + 1003
    x = torch.zeros(M, K, dtype=BF, device=DEV)
    x[:, 3] = (torch.arange(M, device=DEV) % 251 + 1).to(BF)   # whole numbers up to 251, which BF16 holds
    rows = torch.cat([torch.arange(n - 70, n + 70) for n in (70, 1 << 24, first)] + [torch.arange(M - 70, M)]).to(DEV)
    x[rows] = rand(1, len(rows), K)
    codes = torch.full((M, K), 9, dtype=torch.int8, device=DEV)
    q, s = f.quantize_rows_int8(x, codes=codes)
    check_rows(x, q, s, rows)
    q[rows] = 0
    q[rows, 3] = 127
    assert (q[:, 3] == 127).all() and not q[:, :3].any() and not q[:, 4:].any()
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[rows] = False
    want = (x[:, 3].double() / 127).float()
    assert ((s - want).abs() <= 2.0 ** -23 * want)[keep].all()


def test_many_long_rows(f):  # noqa: F811
    """More than 2^22 rows, a workgroup of 1024 threads each: the second launch begins at row 2^22 - 1."""
    first, K = 2 ** 22 - 1, 8208
    M = first + 300
    if torch.cuda.mem_get_info()[0] < 3 * M * K + (20 << 30):
        pytest.skip("takes 103 GB")
    assert first * 1024 < 2 ** 32 <= (first + 1) * 1024
    x = torch.zeros(M, K, dtype=BF, device=DEV)
    rows = torch.cat([torch.arange(0, 5), torch.arange(first - 20, first + 20), torch.arange(M - 5, M)]).to(DEV)
    x[rows] = rand(1, len(rows), K)
    codes = torch.full((M, K), 9, dtype=torch.int8, device=DEV)
    q, s = f.quantize_rows_int8(x, codes=codes)
    check_rows(x, q, s, rows)
    assert int((s != 0).sum()) == len(rows)
    q[rows] = 0
    assert not any(bool(part.any()) for part in q.split(1 << 15))


def test_many_rows_in_a_graph(f):  # noqa: F811
    """Both launches of one call are captured."""
    first = 4 * (2 ** 24 - 1)
    M, K = first + 10, 16
    x = torch.ones(M, K, dtype=BF, device=DEV)
    codes, scales = torch.zeros(M, K, dtype=torch.int8, device=DEV), torch.zeros(M, device=DEV)
    f.quantize_rows_int8(x, codes=codes, scales=scales)
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            f.quantize_rows_int8(x, codes=codes, scales=scales)
    for v in (1, -2, 3):
        x.fill_(v)
        codes.zero_()
        scales.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert (codes == (127 if v > 0 else -127)).all() and (scales == scales[0]).all() and float(scales[0]) > 0
