"""The statistics of rows that hold infinities, wherever these lie in a row: the mean is
their sum's, rstd and Y are NaN, as the formulas have it; the other rows stay."""
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_layer_norm import inputs, run

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("rows,cols", [(8, 64), (8, 72), (8, 512), (8, 520), (8, 1000), (8, 2048), (8, 2056), (8, 5000),
                                       (8, 16384), (8, 16392), (1030, 520), (1030, 4096), (1100, 72), (1030, 5000)])
@pytest.mark.parametrize("x_type", [torch.bfloat16, torch.float32])
def test_statistics_of_rows_with_infinities(rows, cols, x_type):
    need_gpu()
    print("norm infinite", rows, cols, x_type, flush=True)
    X, gamma, beta, _ = inputs(rows, cols, x_type, torch.float32)
    clean = run(X, gamma, beta, 1e-5)
    X[1, 0], X[2, cols // 2], X[3, cols - 1] = INF, -INF, INF
    X[4] = INF                                   # all of it
    X[5, 3], X[5, cols - 2] = INF, -INF          # both: no sum
    X[6, 1], X[6, cols - 1] = INF, INF
    got = run(X, gamma, beta, 1e-5)
    want = torch.tensor([INF, -INF, INF, INF, float("nan"), INF], dtype=torch.float64)
    assert torch.equal(got["mean"][1:7].nan_to_num(nan=7.0, posinf=INF, neginf=-INF),
                       want.nan_to_num(nan=7.0, posinf=INF, neginf=-INF)), got["mean"][1:7]
    assert got["rstd"][1:7].isnan().all() and got["Y"][1:7].isnan().all()
    rest = torch.ones(rows, dtype=torch.bool)
    rest[1:7] = False
    assert all(torch.equal(got[k][rest], clean[k][rest]) for k in got)
