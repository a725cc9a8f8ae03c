"""Cross entropy where logits are large and finite: whole runs of columns masked by
large negative numbers down to BF16's lowest, rows that have nothing else, large
positive logits, and logits around the sizes from which on the kernels compute in
another way; values and gradients against 64 bits, every kernel forced.

The first columns of A and B carry the large part, alone in their row of B, so that
those logits are exact in any order of summation. Bounds, with v = 2^-24, e_z as in
test_gpu_cross_entropy.py, 0 for the exact logits, and s the half-step of a base, the
largest logit times log2(e) (none from 2^30 on, where logits are taken as they are):
  lse   the weights' 6 v d, d the softmax-weighted distance from the row's largest, and
        the sums' v (104 + runs / 16); s in every argument and in the sum's logarithm:
        3 v s; the largest e_z that has a weight; v |lse| for its rounding
  loss  the same with v |loss| (twice: the logarithm's, the result's) for v |lse|, and
        e_z of the target's logit
  dz    p (e_z + 2 v |z - lse| + 6 v + 2 v s), s that of the lse; below EXACT, where the
        base's rounding is not made good, 2 v (|z| + |lse|) p besides; the factors that
        make it good, 8 v of the weight (p and the target's 1 have them)
"""
import pytest
import torch

import dense_gemm_14_amd as g
from tests.dense_util import close
from tests.gpu_util import need_gpu
from tests.rows_util import V as v32, randn
from tests.test_gpu_cross_entropy import KERNELS, U, gen_of, run, run_bwd

pytestmark = pytest.mark.gpu
EXACT = 1024.0
LOWEST = torch.finfo(torch.bfloat16).min
MASKS = [-1e4, -1e9, -1e10, -1e30, -2.4e38, LOWEST, float("-inf")]


def half_step(x):
    """Of x log2(e) rounded to a whole number, at most."""
    return torch.where(x.abs() < 2.0 ** 30, (1.45 * x.abs() * v32).clamp(0.5), 0.5)


def masked(M, V, K, which, values, signs, seed=0):
    """A, B, targets, weights: B's rows `which` hold `values` in column 0 and zeros
    besides, A's column 0 the signs in turn."""
    gen = gen_of(M + V + K + seed)
    A, B = randn(gen, M, K), randn(gen, V, K, std=2 * K ** -0.5)
    B[:, 0] = 0
    B[which] = 0
    B[which, 0] = values.to(torch.bfloat16)
    A[:, 0] = torch.tensor(signs)[torch.arange(M) % len(signs)].to(torch.bfloat16)
    t = torch.randint(0, V, (M,), generator=gen)
    t[::7] = -1
    return A, B, t, torch.randn(M, generator=gen)


def logits(A, B):
    """z and e_z in 64 bits; 0 times infinity, which no kernel is asked for, is left out."""
    a, b = A.double(), B.double()
    exact = (B[:, 1:] == 0).all(1) | (A[:, 1:] == 0).all(1)[:, None]
    inf = torch.isinf(b[:, 0])
    tail = a[:, 1:] @ b[:, 1:].t()
    z = a[:, :1] * torch.where(inf, 0.0, b[:, 0])[None] + tail
    z = torch.where(inf[None], a[:, :1] * b[:, 0][None], z)
    e = (A.shape[1] + 1) * v32 * (a.abs()[:, 1:] @ b.abs()[:, 1:].t())
    return z, torch.where(exact, 0.0, e)


def check_forward(A, B, t):
    z, ez = logits(A, B)
    kept, at = t >= 0, t.clamp(min=0)[:, None]
    top = z.amax(1)
    d = (z - top[:, None]).exp()
    p = d / d.sum(1, keepdim=True)
    spread = (p * torch.nan_to_num(top[:, None] - z, posinf=0.0)).sum(1)
    rest = torch.log(d.sum(1))
    lse, zt = top + rest, z.gather(1, at)[:, 0]
    loss = (top - zt) + rest
    e = v32 * (6 * spread + 104 + B.shape[0] / 16 / 16 + 3 * half_step(top)) + torch.where(p > 0, ez, 0.0).amax(1)
    e_lse = e + v32 * lse.abs()
    e_loss = e + ez.gather(1, at)[:, 0] + 2 * v32 * loss.abs()
    nil = torch.zeros_like(lse)
    got = run(A, B, t)
    for k, (x, y) in {"lse": (lse, e_lse), "loss": (loss, e_loss)}.items():
        # (what lies beyond FP32 rounds to infinity)
        x = torch.where(x.abs() > torch.finfo(torch.float32).max, x * float("inf"), x)
        y = torch.where(torch.isfinite(x), y, nil)
        same = kept & ~torch.isfinite(x)
        assert torch.equal(got[k][same], x[same]), k
        close(torch.where(same, nil, got[k]), torch.where(kept & ~same, x, nil), torch.where(kept & ~same, y, nil), k)
    return torch.where(kept, lse, nil).float()


def weight_error(z, l, ez):
    """Relative error of exp(z - l) as the kernels compute it."""
    apart = torch.nan_to_num((z - l).abs(), posinf=0.0)
    small = torch.where(l.abs() < EXACT, torch.nan_to_num(z, neginf=0.0).abs() + l.abs(), half_step(l))
    return ez + v32 * (2 * apart + 6 + 2 * small)


def check_gradients(A, B, t, lse, w):
    """lse as it was rounded, which the formula takes as given."""
    z, ez = logits(A, B)
    kept, at = (t >= 0)[:, None], t.clamp(min=0)[:, None]
    l, w = lse.double()[:, None], torch.where(kept, w.double()[:, None], 0.0)
    p = torch.where(kept, torch.exp(z - l), 0.0)
    one = torch.zeros_like(p).scatter_(1, at, 1.0)
    e = p * weight_error(z, l, ez)
    e = torch.where(p > 0, e, 0.0) * w.abs()
    dz = (p - one) * w
    e = e + 8 * v32 * (p + one) * w.abs()
    e = torch.where(kept, e + U * (dz.abs() + e) + 1e-37, 0.0)

    def prod(x, ex, y):
        out = x @ y
        err = ex @ y.abs() + (x.shape[1] + 2) * v32 * ((x.abs() + ex) @ y.abs())
        return out, err + U * (out.abs() + err)
    a = torch.where(kept, A.double(), 0.0)
    # (dA's first column is as large as the masks: a sum of values that differ by forty
    # orders of magnitude, compared where no mask is a target)
    got = run_bwd(A, B, t, lse, w[:, 0].float())
    close(got["dB"], *prod(dz.t().contiguous(), e.t().contiguous(), a), "dB")
    out, err = prod(dz, e, torch.nan_to_num(B.double()[:, 1:]))
    close(got["dA"][:, 1:], out, err, "dA")


def forced(kernel, f):
    g.force_layer_kernel(kernel)
    try:
        f()
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)


SIZES = [(5, 700, 72), (70, 1100, 264), (300, 1031, 520)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,V,K", SIZES)
@pytest.mark.parametrize("mask", MASKS)
def test_masked_runs(M, V, K, mask, kernel):
    # the last 300 ids and 260 in the middle; rows with the mask, without it and, where
    # it is finite, with its opposite: a large positive logit in every run
    need_gpu()
    print("ce masked", M, V, K, mask, kernel, flush=True)
    which = torch.cat([torch.arange(128, 388), torch.arange(V - 300, V)])
    finite = mask != float("-inf")
    A, B, t, w = masked(M, V, K, which, torch.full((len(which),), mask), [1.0, 0.0, -1.0, 1.0] if finite else [1.0])

    def both():
        lse = check_forward(A, B, t)
        if finite:      # (an infinite row of B is one in the products as well: 0 times infinity)
            check_gradients(A, B, t, lse, w)
    forced(kernel, both)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,V,K", SIZES)
def test_runs_masked_by_different_values(M, V, K, kernel):
    need_gpu()
    print("ce masks", M, V, K, kernel, flush=True)
    which = torch.arange(0, V - 9)
    values = torch.tensor(MASKS[:-1])[which // 64 % (len(MASKS) - 1)]
    A, B, t, w = masked(M, V, K, which, values, [1.0, -1.0, 0.5, -0.25])
    forced(kernel, lambda: check_gradients(A, B, t, check_forward(A, B, t), w))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,V,K", SIZES)
@pytest.mark.parametrize("value", [-1e4, 1e6, -1e10, 1e10, -1e30, 3e38, LOWEST, -LOWEST])
def test_every_logit_is_large(M, V, K, value, kernel):
    # all the same: loss log V; then neighbours of that value, and with everything else
    # in a row of A zero
    need_gpu()
    print("ce all large", M, V, K, value, kernel, flush=True)
    for steps in (0, 3):
        values = torch.full((V,), value) * (1 - 2.0 ** -7 * (torch.arange(V) * 5 % (steps + 1)))
        A, B, t, w = masked(M, V, K, torch.arange(V), values, [1.0, 0.5])

        def both():
            lse = check_forward(A, B, t)
            if steps == 0 and abs(value) > 1e9:
                z = logits(A, B)[0]
                assert torch.equal(lse[t >= 0].double(), z[t >= 0, 0].float().double())    # log V is less than a step
            check_gradients(A, B, t, lse, w)
        forced(kernel, both)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("size,step", [(2.0 ** 9, 1), (2.0 ** 10, 1), (2.0 ** 11, 1), (2.0 ** 20, 1), (2.0 ** 22, 1),
                                       (2.0 ** 27, 16), (2.0 ** 30, 128), (2.0 ** 31, 256), (2.0 ** 40, 2.0 ** 17)])
def test_around_a_limit(size, step, kernel):
    # logits +-size + x, x whole and from -6 to 6 steps, in runs of one x: some runs lie
    # on either side of a limit that is a power of two. All weigh, or (from 2^27 on) those
    # of the largest x
    need_gpu()
    print("ce limit", size, kernel, flush=True)
    M, V, K = 90, 1400, 72
    for sign in (1.0, -1.0):
        B, A = torch.zeros(V, K, dtype=torch.bfloat16), torch.zeros(M, K, dtype=torch.bfloat16)
        B[:, 0] = size * sign
        B[:, 1] = step * (torch.arange(V) // 16 * 5 % 13 - 6).to(torch.bfloat16)
        A[:, 0] = 1
        A[:, 1] = torch.tensor([1.0, -1.0, 0.0])[torch.arange(M) % 3].to(torch.bfloat16)
        t = torch.randint(-1, V, (M,), generator=gen_of(3))
        w = torch.randn(M, generator=gen_of(4))

        def both():
            z = A.double() @ B.double().t()      # exact in FP32
            lse = check_limit(z, A, B, t)
            got = run_bwd(A, B, t, lse, w)
            kept, at = (t >= 0)[:, None], t.clamp(min=0)[:, None]
            l = lse.double()[:, None]
            p = torch.where(kept, torch.exp(z - l), 0.0)
            one, wd = torch.zeros_like(p).scatter_(1, at, 1.0) * kept, w.double()[:, None]
            dz = (p - one) * wd
            e = (p * weight_error(z, l, 0.0) + 8 * v32 * (p + one)) * wd.abs()
            e = e + U * (dz.abs() + e) + 1e-37
            a = torch.where(kept, A.double(), 0.0)
            out, err = dz.t() @ a, e.t() @ a.abs() + (M + 2) * v32 * (dz.abs().t() @ a.abs())
            close(got["dB"], out, err + U * (out.abs() + err), "dB")
        forced(kernel, both)


def check_limit(z, A, B, t):
    top = z.amax(1)
    rest = torch.log((z - top[:, None]).exp().sum(1))
    zt = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    kept, lse, loss = t >= 0, top + rest, top - zt + rest
    p = (z - lse[:, None]).exp()
    e = v32 * (6 * (p * (top[:, None] - z)).sum(1) + 104 + len(B) / 256 + 3 * half_step(top))
    nil, got = torch.zeros_like(lse), run(A, B, t)
    close(got["lse"], torch.where(kept, lse, nil), torch.where(kept, e + v32 * lse.abs(), nil), "lse")
    close(got["loss"], torch.where(kept, loss, nil), torch.where(kept, e + 2 * v32 * loss.abs(), nil), "loss")
    return torch.where(kept, lse, nil).float()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,V,K", SIZES)
def test_infinity_and_nan_beside_masks(M, V, K, kernel):
    # one logit in another run than masks of either sign: infinite, or NaN
    need_gpu()
    print("ce not finite", M, V, K, kernel, flush=True)
    which = torch.arange(128, V)
    A, B, t, _ = masked(M, V, K, which, torch.tensor([LOWEST, 1e30, -1e10])[which // 128 % 3], [1.0])
    t[t == 5] = 6
    t[1] = 5
    for value in (float("inf"), float("nan")):
        B[5] = 0
        B[5, 0] = value
        out = {}
        forced(kernel, lambda: out.update(run(A, B, t)))
        kept, nan = t >= 0, torch.arange(M) == 1
        if value == float("inf"):
            assert (out["lse"][kept] == value).all() and (out["loss"][kept & ~nan] == value).all()
            assert out["loss"][1].isnan()
        else:
            assert out["lse"][kept].isnan().all() and out["loss"][kept].isnan().all()
        assert (out["lse"][~kept] == 0).all() and (out["loss"][~kept] == 0).all()
