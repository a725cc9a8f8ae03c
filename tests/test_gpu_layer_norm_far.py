"""Layer norm of rows so far from zero that their mean's square, or the mean in units of
their spread, lies beyond FP32. Statistics and gradients against 64 bits, at widths that
fill the lanes of a row, leave some of them empty and leave whole waves empty."""
import pytest
import torch

from tests.dense_util import close
from tests.gpu_util import need_gpu
from tests.rows_util import V as v32, norm_bwd, randn
from tests.test_gpu_layer_norm import check, gen_of, run, run_bwd

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
WIDTHS = [(3, 64), (3, 72), (5, 512), (3, 520), (2, 1000), (2, 2048), (3, 2056), (2, 5000), (2, 8200), (2, 16392),
          (1030, 520), (1030, 1000), (1030, 4096), (1100, 72)]


@pytest.mark.parametrize("rows,cols", WIDTHS)
@pytest.mark.parametrize("x_type", [BF16, FP32])
def test_statistics_of_rows_far_from_zero(rows, cols, x_type):
    # constant rows of 2^70 (their squares are beyond FP32): sums of up to 16392 equal
    # powers of two round nowhere if their number is a power of two, else to 2^-24 of
    # the mean at each of (96 + cols / 8192) additions
    need_gpu()
    print("norm far", rows, cols, x_type, flush=True)
    X = torch.full((rows, cols), 2.0 ** 70).to(x_type)
    X[1::2] = -X[1::2]
    got = run(X, None, None, 1e-5)
    x = X[:, 0].double()
    e = (97 + cols // 8192) * v32 * x.abs()
    close(got["mean"], x, e, "mean")
    # rstd: 1 / sqrt(eps) if the mean is exact; with a mean that is off by e, the
    # difference squared under the root. Never NaN, never negative.
    eps = torch.tensor(1e-5).double()
    assert (got["rstd"] <= 1 / torch.sqrt(eps) * (1 + 8 * v32)).all()
    low = 1 / torch.sqrt(eps + 4 * e ** 2)
    assert (got["rstd"] >= low * (1 - 8 * v32)).all()
    # |y| = |x - mean| rstd: at most 1, as of any constant row whose mean is off
    assert torch.isfinite(got["Y"]).all() and (got["Y"].abs() <= 1 + 2.0 ** -7).all()


@pytest.mark.parametrize("rows,cols", WIDTHS)
@pytest.mark.parametrize("x_type", [BF16, FP32])
def test_gradients_of_rows_far_from_zero(rows, cols, x_type):
    # every second row constant at +-2^110, with the rstd of eps = 2^-38: mean times rstd
    # is 2^129, beyond FP32, and (x - mean) rstd is 0
    need_gpu()
    print("norm_bwd far", rows, cols, x_type, flush=True)
    gen = gen_of(rows + cols)
    X = torch.randn(rows, cols, generator=gen).to(x_type)
    mean, rstd = X.double().mean(1).float(), (1 / X.double().std(1, correction=0)).float()
    X[::2], mean[::2], rstd[::2] = 2.0 ** 110, 2.0 ** 110, 2.0 ** 19
    X[::4], mean[::4] = -2.0 ** 110, -2.0 ** 110
    dY, R = randn(gen, rows, cols), randn(gen, rows, cols, dtype=x_type)
    gamma = randn(gen, cols, dtype=FP32)
    check(run_bwd(X, gamma, mean, rstd, dY, R, FP32), norm_bwd(X, gamma, mean, rstd, dY, R, FP32))
