"""Layer norm and its gradients against 64-bit references on the GPU: every type,
widths of every kernel, single rows and many, missing outputs, rows that are far
off centre, constant or hold infinities, repeatability."""
import pytest
import torch

import dense_gemm_14_amd as g
from tests.dense_util import close
from tests.gpu_util import need_gpu
from tests.rows_util import Array, norm, norm_bwd, randn

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (FP32, FP32), (FP32, BF16), (BF16, FP32)]
SIZES = [(1, 8), (1, 64), (3, 72), (2, 512), (5, 520), (1, 1000), (1, 4096), (7, 1032), (9, 2056), (3, 5000), (2, 8200),
         (3, 16384), (2, 16392), (2, 32776), (1030, 8), (1111, 72), (1025, 520), (1100, 1544), (1030, 4096), (300, 2048),
         (261, 5000), (270, 8200), (259, 16384),
         (1, 136), (5, 256), (2003, 64), (9000, 128), (4099, 136), (1037, 256), (1029, 264), (805, 136),
         (800, 1000), (801, 8), (801, 1000), (820, 3000), (900, 5000), (801, 8192), (803, 8200), (805, 16384)]


def gen_of(seed):
    gen = torch.Generator()
    gen.manual_seed(seed)
    return gen


def inputs(rows, cols, x_type, w_type):
    gen = gen_of(rows * 7 + cols)
    size = torch.exp(torch.randn(rows, 1, generator=gen))
    X = ((torch.randn(rows, cols, generator=gen) + 0.5) * size).to(x_type)
    return X, randn(gen, cols, dtype=w_type), randn(gen, cols, dtype=w_type), gen


def dev(x):
    return None if x is None else x.cuda()


def run(X, gamma, beta, eps, want=("Y", "mean", "rstd")):
    rows, cols = X.shape
    outs = {"Y": Array(rows, cols), "mean": Array(rows, dtype=FP32), "rstd": Array(rows, dtype=FP32)}
    g.layer_norm(rows, cols, dev(X), dev(gamma), dev(beta), *[outs[k].t if k in want else None for k in outs], eps)
    torch.cuda.synchronize()
    return {k: outs[k].get() for k in want}


def run_bwd(X, gamma, mean, rstd, dY, R, wtype, want=("dX", "dgamma", "dbeta"), in_place=False):
    rows, cols = X.shape
    outs = {"dX": Array(rows, cols, dtype=X.dtype, fill=R if in_place else None), "dgamma": Array(cols, dtype=wtype),
            "dbeta": Array(cols, dtype=wtype)}
    nb = g.layer_norm_bwd_workspace_size(rows, cols)
    ws = torch.full((nb + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    g.layer_norm_bwd(rows, cols, dev(X), dev(gamma), dev(mean), dev(rstd), dev(dY), outs["dX"].t if in_place else dev(R),
                     *[outs[k].t if k in want else None for k in outs], ws, nb)
    torch.cuda.synchronize()
    assert (ws[nb:] == 0xFF).all(), "write past the workspace"
    return {k: outs[k].get() for k in want}


def check(got, want):
    for k in got:
        close(got[k], *want[k], k)


@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols):
    need_gpu()
    for i, (x_type, w_type) in enumerate(TYPES):
        print("norm", rows, cols, x_type, w_type, flush=True)
        X, gamma, beta, _ = inputs(rows, cols, x_type, w_type)
        if i == 1:
            gamma = None
        if i == 2:
            beta = None
        check(run(X, gamma, beta, 1e-5), norm(X, gamma, beta, 1e-5))


@pytest.mark.parametrize("rows,cols", SIZES)
def test_gradients(rows, cols):
    need_gpu()
    for i, (x_type, w_type) in enumerate(TYPES):
        print("norm_bwd", rows, cols, x_type, w_type, flush=True)
        X, gamma, _, gen = inputs(rows, cols, x_type, w_type)
        dY = randn(gen, rows, cols)
        R = randn(gen, rows, cols, dtype=x_type) if i != 1 else None
        gamma = None if i == 3 else gamma
        st = norm(X, None, None, 1e-5)
        mean, rstd = st["mean"][0].float(), st["rstd"][0].float()
        want = norm_bwd(X, gamma, mean, rstd, dY, R, w_type)
        check(run_bwd(X, gamma, mean, rstd, dY, R, w_type, in_place=i == 2), want)


@pytest.mark.parametrize("rows,cols", [(3, 72), (300, 520), (290, 5000), (2, 16392)])
def test_outputs_that_are_not_wanted(rows, cols):
    need_gpu()
    X, gamma, beta, gen = inputs(rows, cols, FP32, FP32)
    dY = randn(gen, rows, cols)
    full = run(X, gamma, beta, 1e-5)
    mean, rstd = full["mean"].float(), full["rstd"].float()
    for want in (("Y",), ("Y", "mean"), ("Y", "rstd")):
        got = run(X, gamma, beta, 1e-5, want)
        assert all(torch.equal(got[k], full[k]) for k in want)
    back = run_bwd(X, gamma, mean, rstd, dY, None, FP32)
    for want in (("dX",), ("dgamma",), ("dbeta",), ("dX", "dbeta"), ("dgamma", "dbeta")):
        got = run_bwd(X, gamma, mean, rstd, dY, None, FP32, want)
        assert all(torch.equal(got[k], back[k]) for k in want), want


def test_no_rows_give_zero_gradients():
    need_gpu()
    dg, db = Array(72, dtype=FP32), Array(72)
    e = torch.zeros(0, 72, dtype=BF16, device="cuda")
    n = torch.zeros(0, device="cuda")
    g.layer_norm_bwd(0, 72, e, None, n, n, e, None, e, dg.t, None)
    g.layer_norm_bwd(0, 72, e, None, n, n, e, None, e, None, db.t)
    torch.cuda.synchronize()
    assert (dg.get() == 0).all() and (db.get() == 0).all()


@pytest.mark.parametrize("cols", [64, 1032, 5000, 16392])
def test_rows_that_are_hard(cols):
    # far off centre (the squares' mean would cancel), constant, tiny, huge, zero
    need_gpu()
    gen = gen_of(cols)
    X = torch.randn(6, cols, generator=gen)
    X[0] += 1000
    X[1] = 3.0
    X[2] *= 1e-12
    X[3] *= 1e15
    X[4] = 0
    X[5, 3:] = 0
    for eps in (1e-5, 1e-12):
        check(run(X, None, None, eps), norm(X, None, None, eps))
    # eps 0 where the variance is not
    check(run(X[[0, 3, 5]], None, None, 0.0), norm(X[[0, 3, 5]], None, None, 0.0))


@pytest.mark.parametrize("rows,cols", [(9, 72), (1100, 64), (900, 136), (1100, 520), (6, 5000), (3, 16392)])
def test_infinities_stay_in_their_row(rows, cols):
    need_gpu()
    X, gamma, beta, gen = inputs(rows, cols, BF16, BF16)
    clean = run(X, gamma, beta, 1e-5)
    bad = X.clone()
    bad[1, 5] = float("inf")
    bad[2, cols - 1] = float("nan")
    got = run(bad, gamma, beta, 1e-5)
    ok = torch.ones(rows, dtype=torch.bool)
    ok[1:3] = False
    assert all(torch.equal(got[k][ok], clean[k][ok]) for k in got)
    assert got["Y"][2].isnan().all() and got["Y"][1].isnan().any()
    dY = randn(gen, rows, cols)
    mean, rstd = clean["mean"].float(), clean["rstd"].float()
    a, b = (run_bwd(x, gamma, mean, rstd, dY, None, BF16, ("dX",))["dX"] for x in (X, bad))
    assert torch.equal(a[ok], b[ok]) and b[2].isnan().all()


def test_gradients_are_the_same_every_time():
    need_gpu()
    for rows, cols in ((2000, 1032), (200, 1032), (500, 5000)):
        X, gamma, _, gen = inputs(rows, cols, FP32, FP32)
        dY, st = randn(gen, rows, cols), norm(X, None, None, 1e-5)
        args = (X, gamma, st["mean"][0].float(), st["rstd"][0].float(), dY, None, FP32)
        first = run_bwd(*args)
        for _ in range(4):
            again = run_bwd(*args)
            assert all(torch.equal(first[k], again[k]) for k in first)


def test_gradients_against_differences():
    # of the reference's own forward formula in 64 bits, along random directions
    need_gpu()
    rows, cols, eps, h = 5, 72, 1e-5, 1e-6
    X, gamma, beta, gen = inputs(rows, cols, FP32, FP32)
    dY = randn(gen, rows, cols)
    st = run(X, gamma, beta, eps)
    got = run_bwd(X, gamma, st["mean"].float(), st["rstd"].float(), dY, None, FP32)

    def loss(x, w, b):
        m = x.mean(1, keepdim=True)
        v = ((x - m) ** 2).mean(1, keepdim=True)
        return (((x - m) / torch.sqrt(v + eps) * w + b) * dY.double()).sum()
    base = [X.double(), gamma.double(), beta.double()]
    for i, k in enumerate(("dX", "dgamma", "dbeta")):
        for _ in range(4):
            d = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
            up, down = ([b + s * h * d if j == i else b for j, b in enumerate(base)] for s in (1, -1))
            slope = (loss(*up) - loss(*down)) / (2 * h)
            # the difference's own error: h^2 of the third derivative and 2^-52 of
            # the loss over h, about 1e-8; the gradient's: 2^-24 of its terms, times
            # the 100 additions of a row
            size = (got[k] * d).abs().sum()
            assert abs(slope - (got[k] * d).sum()) <= 1e-5 * size + 1e-5, (k, slope)


def test_far_offsets():
    # arrays of more than 2^32 bytes: the last rows as the first
    need_gpu()
    rows, cols = 600000, 4096
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    X = torch.randn(64, cols, generator=gen, device="cuda").bfloat16().repeat(rows // 64, 1)
    Y, mean, rstd = torch.empty_like(X), *(torch.empty(rows, device="cuda") for _ in range(2))
    g.layer_norm(rows, cols, X, None, None, Y, mean, rstd)
    assert torch.equal(Y.view(-1, 64 * cols)[0], Y.view(-1, 64 * cols)[-1])
    assert torch.equal(mean.view(-1, 64), mean[:64].expand(rows // 64, 64))
    dX, dg = torch.empty_like(X), torch.empty(cols, dtype=BF16, device="cuda")
    ws = torch.empty(g.layer_norm_bwd_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    g.layer_norm_bwd(rows, cols, X, None, mean, rstd, Y, None, dX, dg, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(dX.view(-1, 64 * cols)[0], dX.view(-1, 64 * cols)[-1])
    st = norm_bwd(X[:64].cpu(), None, mean[:64].cpu(), rstd[:64].cpu(), Y[:64].cpu(), None, BF16)
    close(dX[-64:].cpu().double(), *st["dX"], "dX")
