"""The layer calls against 64-bit references on the GPU: linear and gated
layers forward and backward, every activation, ragged sizes, empty sums, the
residual in place, split K, exact sums bitwise, and a block of them run
together."""
import pytest
import torch

import dense_gemm_14_amd as g
from tests.dense_util import Out, act, backward, close, forward, ints, randn, workspace
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
ACTS = [g.ACT_NONE, g.ACT_RELU, g.ACT_GELU_TANH, g.ACT_SILU]


def gen_of(*key):
    gen = torch.Generator()
    gen.manual_seed(hash(key) % (1 << 31))
    return gen


def dev(x):
    return None if x is None else x.cuda()


def run_forward(gated, M, N, K, A, B, bias, name, R, want_z, in_place=False):
    rows = 2 * N if gated else N
    C = Out(M, N, fill=dev(R) if in_place else None)
    Z = Out(M, rows) if want_z else None
    ws, nb, check = workspace(g.gated_workspace_size(M, N, K) if gated else g.bias_act_res_workspace_size(M, N, K))
    if gated:
        g.gemm_bf16_nt_gated(M, N, K, dev(A), dev(B), dev(bias), name, Z.t if Z else None, C.t, ws, nb)
    else:
        g.gemm_bf16_nt_bias_act_res(M, N, K, dev(A), dev(B), dev(bias), name, C.t if in_place else dev(R),
                                    Z.t if Z else None, C.t, ws, nb)
    torch.cuda.synchronize()
    check()
    return C.get(), Z.get() if Z else None


def run_backward(gated, M, N, K, A, B, Z, name, dC, want=("dA", "dB", "dbias")):
    rows = 2 * N if gated else N
    outs = {"dA": Out(M, K), "dB": Out(rows, K), "dbias": Out(rows)}
    nb = g.gated_bwd_workspace_size(M, N, K) if gated else g.bias_act_bwd_workspace_size(M, N, K, name)
    ws, nb, check = workspace(nb)
    call = g.gemm_bf16_nt_gated_bwd if gated else g.gemm_bf16_nt_bias_act_bwd
    call(M, N, K, dev(A), dev(B), dev(Z), name, dev(dC), *[outs[k].t if k in want else None for k in outs], ws, nb)
    torch.cuda.synchronize()
    check()
    return {k: outs[k].get() for k in want}


SIZES = [(1, 8, 8), (1, 264, 1032), (3, 128, 64), (16, 72, 520), (17, 136, 72), (65, 72, 64), (130, 200, 264),
         (300, 264, 520), (129, 1384, 2056)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_forward_matches_64_bits(gated, M, N, K):
    need_gpu()
    rows = 2 * N if gated else N
    for name in ACTS:
        gen = gen_of(M, N, K, name)
        A, B = randn(gen, M, K), randn(gen, rows, K, std=K ** -0.5)
        bias = randn(gen, rows, std=0.5) if name != g.ACT_RELU else None
        R = randn(gen, M, N) if not gated and name != g.ACT_SILU else None
        print("forward", gated, M, N, K, name, flush=True)
        C, Z = run_forward(gated, M, N, K, A, B, bias, name, R, want_z=name != g.ACT_NONE)
        y, ey, z, ez = forward(A, B, bias, name, R, gated)
        close(C, y, ey, "C")
        if Z is not None:
            close(Z, z, ez, "Z")


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_backward_matches_64_bits(gated, M, N, K):
    need_gpu()
    rows = 2 * N if gated else N
    for name in ACTS:
        gen = gen_of(M, N, K, name, 1)
        A, B = randn(gen, M, K), randn(gen, rows, K, std=K ** -0.5)
        Z, dC = randn(gen, M, rows, std=2.0), randn(gen, M, N, std=2.0 ** -8)
        print("backward", gated, M, N, K, name, flush=True)
        got = run_backward(gated, M, N, K, A, B, Z if gated or name else None, name, dC)
        for k, (v, e) in backward(A, B, Z, name, dC, gated).items():
            close(got[k], v, e, k)


@pytest.mark.parametrize("M,N,K", [(130, 200, 264), (513, 520, 136), (64, 4096, 520), (1100, 136, 1032)])
def test_whole_numbers_are_exact(M, N, K):
    # every sum is exact in FP32, so each output has one right value
    need_gpu()
    gen = gen_of(M, N, K, 2)
    A, B, R, bias, dC = ints(gen, M, K), ints(gen, N, K), ints(gen, M, N), ints(gen, N), ints(gen, M, N)
    C, Z = run_forward(False, M, N, K, A, B, bias, g.ACT_RELU, R, True)
    z = A.double() @ B.double().t() + bias.double()
    assert torch.equal(Z, z.bfloat16().double())
    assert torch.equal(C, (z.clamp(min=0) + R.double()).bfloat16().double())
    got = run_backward(False, M, N, K, A, B, None, g.ACT_NONE, dC)
    d = dC.double()
    assert torch.equal(got["dA"], (d @ B.double()).bfloat16().double())
    assert torch.equal(got["dB"], (d.t().contiguous() @ A.double()).bfloat16().double())
    assert torch.equal(got["dbias"], d.sum(0).bfloat16().double())
    if N % 16 == 0:
        n = N // 2
        C, Z = run_forward(True, M, n, K, A, B, bias, g.ACT_RELU, None, True)
        assert torch.equal(Z, z.bfloat16().double())
        assert torch.equal(C, (z[:, :n].clamp(min=0).float() * z[:, n:].float()).bfloat16().double())


def test_residual_in_place_and_split_k():
    need_gpu()
    M, N, K = 40, 136, 4104      # one row of tiles and a long K: split
    gen = gen_of(7)
    A, B, R = randn(gen, M, K), randn(gen, N, K, std=K ** -0.5), randn(gen, M, N)
    want = run_forward(False, M, N, K, A, B, None, g.ACT_GELU_TANH, R, False)[0]
    got = run_forward(False, M, N, K, A, B, None, g.ACT_GELU_TANH, R, False, in_place=True)[0]
    assert torch.equal(want, got)
    y, ey, _, _ = forward(A, B, None, g.ACT_GELU_TANH, R, False)
    close(got, y, ey, "C")


@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_empty_sums(gated):
    need_gpu()
    gen = gen_of(11)
    M, N = 37, 72
    rows = 2 * N if gated else N
    # K = 0: the pre-activations are the bias
    bias = randn(gen, rows)
    R = None if gated else randn(gen, M, N)
    A, B = torch.zeros(M, 0, dtype=torch.bfloat16), torch.zeros(rows, 0, dtype=torch.bfloat16)
    C, Z = run_forward(gated, M, N, 0, None, None, bias, g.ACT_SILU, R, True)
    y, ey, z, _ = forward(A, B, bias, g.ACT_SILU, R, gated)
    close(C, y, ey, "C")
    assert torch.equal(Z, z)
    # M = 0: sums over no tokens
    got = run_backward(gated, 0, N, 40, None, None, None, g.ACT_RELU, None, want=("dB", "dbias"))
    assert not got["dB"].any() and not got["dbias"].any()
    # N = 0: sums over no outputs
    got = run_backward(gated, M, 0, 40, None, None, None, g.ACT_RELU, None, want=("dA",))
    assert not got["dA"].any()


def test_only_the_wanted_gradients():
    need_gpu()
    M, N, K = 70, 136, 200
    gen = gen_of(13)
    A, B, Z, dC = randn(gen, M, K), randn(gen, N, K), randn(gen, M, N), randn(gen, M, N)
    every = run_backward(False, M, N, K, A, B, Z, g.ACT_GELU_TANH, dC)
    for k in every:
        one = run_backward(False, M, N, K, A if k == "dB" else None, B if k == "dA" else None, Z, g.ACT_GELU_TANH, dC,
                           want=(k,))
        assert torch.equal(one[k], every[k]), k


def test_gradients_against_differences():
    # the sum of C weighted by dC, moved along a direction of each input
    need_gpu()
    M, N, K = 33, 40, 48
    gen = gen_of(17)
    for gated in (False, True):
        rows = 2 * N if gated else N
        A, B, bias = randn(gen, M, K), randn(gen, rows, K, std=K ** -0.5), randn(gen, rows)
        dC = randn(gen, M, N)
        _, Z = run_forward(gated, M, N, K, A, B, bias, g.ACT_SILU, None, True)
        got = run_backward(gated, M, N, K, A, B, Z.bfloat16(), g.ACT_SILU, dC)
        a, b, c, d = A.double(), B.double(), bias.double(), dC.double()

        def loss(a, b, c):
            z = a @ b.t() + c
            y = act(g.ACT_SILU, z[:, :N]) * z[:, N:] if gated else act(g.ACT_SILU, z)
            return (y * d).sum()
        h = 1e-5
        for k, x in (("dA", a), ("dB", b), ("dbias", c)):
            t = torch.randn(x.shape, generator=gen, dtype=torch.float64)
            moved = lambda step: loss(*[v + step * t if v is x else v for v in (a, b, c)])
            diff = (moved(h) - moved(-h)) / (2 * h)
            # every element of the gradient is off by a few half-steps at most
            # (Z, dZ and its own rounding): their sum along t by its 2-norm
            scale = (got[k] * t).norm() + got[k].norm()
            assert abs((got[k] * t).sum() - diff) <= 8 * 2.0 ** -8 * scale, (gated, k)


def ortho_exact(G, steps, coef, eps):
    a, b, c = coef
    x = G.double()
    x = x / (x.flatten(1).norm(dim=1)[:, None, None] + eps)
    out = []
    for m in x:
        t = m if m.shape[0] <= m.shape[1] else m.t()
        for _ in range(steps):
            s = t @ t.t()
            t = a * t + (b * s + c * s @ s) @ t
        out.append(t if m.shape[0] <= m.shape[1] else t.t())
    return torch.stack(out)


def run_ortho(G, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7):
    b, r, c = G.shape
    O = Out(b, r, c)
    ws, nb, check = workspace(g.newton_schulz_workspace_size(b, r, c))
    g.newton_schulz(b, r, c, G.cuda(), O.t, steps, coef, eps, ws, nb)
    torch.cuda.synchronize()
    check()
    return O.get()


@pytest.mark.parametrize("shape", [(1, 8, 8), (2, 64, 64), (3, 72, 200), (1, 264, 136), (2, 256, 1032), (1, 520, 392),
                                   (1, 16, 2056)])
@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
def test_newton_schulz(shape, fp32):
    need_gpu()
    gen = gen_of(*shape)
    G = torch.randn(*shape, generator=gen, dtype=torch.float64) * 1e-3
    G = G.float() if fp32 else G.bfloat16()
    print("ortho", shape, fp32, flush=True)
    got, want = run_ortho(G), ortho_exact(G, 5, (3.4445, -4.7750, 2.0315), 1e-7)
    # three roundings to FP16 (2^-11 at most, 2^-11 / sqrt(3) in the mean
    # square) in each of five steps, each step's errors carried on by a slope
    # of about one, plus the BF16 rounding of the result (2^-8 / sqrt(3))
    rel = ((got - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max().item()
    assert rel <= 15 ** 0.5 * 2.0 ** -11 * 2 + 2.0 ** -8 / 3 ** 0.5, rel


def test_newton_schulz_extremes():
    need_gpu()
    gen = gen_of(23)
    G = torch.randn(2, 64, 136, generator=gen)
    base = run_ortho(G, eps=0.0)
    # the norm is taken in FP64 and the scales are powers of two: the same
    # bits for gradients whose squares leave FP32's range
    assert torch.equal(run_ortho(G * 2.0 ** -100, eps=0.0), base)
    assert torch.equal(run_ortho(G * 2.0 ** 100, eps=0.0), base)
    G[1] = 0.0     # a zero matrix beside another
    got = run_ortho(G, eps=0.0)
    assert not got[1].any() and torch.equal(got[0], base[0])
    # one step of the identity map: X = G / |G|
    one = run_ortho(G, steps=1, coef=(1.0, 0.0, 0.0), eps=0.0)
    want = G[0].double() / G[0].double().norm()
    assert ((one[0] - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want.abs() + 2.0 ** -24).all()


def test_feed_forward_block_runs_together():
    # a gated layer, a projection with its residual, both backward passes and
    # the updates of both weights, on one stream with one workspace
    need_gpu()
    M, D, F = 150, 136, 264
    gen = gen_of(29)
    X, W1, W2 = randn(gen, M, D), randn(gen, 2 * F, D, std=D ** -0.5), randn(gen, D, F, std=F ** -0.5)
    dY = randn(gen, M, D, std=2.0 ** -6)
    need = max(g.gated_workspace_size(M, F, D), g.bias_act_res_workspace_size(M, D, F),
               g.bias_act_bwd_workspace_size(M, D, F, g.ACT_NONE), g.gated_bwd_workspace_size(M, F, D),
               g.newton_schulz_workspace_size(1, 2 * F, D), g.newton_schulz_workspace_size(1, D, F))
    ws, nb, check = workspace(need)
    x, w1, w2, dy = dev(X), dev(W1), dev(W2), dev(dY)
    H, Z, Y = Out(M, F), Out(M, 2 * F), Out(M, D)
    dH, dW2, dX, dW1 = Out(M, F), Out(D, F), Out(M, D), Out(2 * F, D)
    U1, U2 = Out(2 * F, D), Out(D, F)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        g.gemm_bf16_nt_gated(M, F, D, x, w1, None, g.ACT_SILU, Z.t, H.t, ws, nb)
        g.gemm_bf16_nt_bias_act_res(M, D, F, H.t, w2, None, g.ACT_NONE, x, None, Y.t, ws, nb)
        g.gemm_bf16_nt_bias_act_bwd(M, D, F, H.t, w2, None, g.ACT_NONE, dy, dH.t, dW2.t, None, ws, nb)
        g.gemm_bf16_nt_gated_bwd(M, F, D, x, w1, Z.t, g.ACT_SILU, dH.t, dX.t, dW1.t, None, ws, nb)
        g.newton_schulz(1, 2 * F, D, dW1.t, U1.t, workspace=ws, workspace_bytes=nb)
        g.newton_schulz(1, D, F, dW2.t, U2.t, workspace=ws, workspace_bytes=nb)
    torch.cuda.synchronize()
    check()
    # each call against its reference on the inputs it was given
    h, z = H.get().bfloat16(), Z.get().bfloat16()
    y, ey, zz, ez = forward(X, W1, None, g.ACT_SILU, None, True)
    close(H.get(), y, ey, "H")
    close(Z.get(), zz, ez, "Z")
    y, ey, _, _ = forward(h, W2, None, g.ACT_NONE, X, False)
    close(Y.get(), y, ey, "Y")
    r = backward(h, W2, None, g.ACT_NONE, dY, False)
    close(dH.get(), *r["dA"], "dH")
    close(dW2.get(), *r["dB"], "dW2")
    r = backward(X, W1, z, g.ACT_SILU, dH.get().bfloat16(), True)
    close(dX.get(), *r["dA"], "dX")
    close(dW1.get(), *r["dB"], "dW1")
    for O, G in ((U1, dW1), (U2, dW2)):
        want = ortho_exact(G.get()[None], 5, (3.4445, -4.7750, 2.0315), 1e-7)[0]
        # as in test_newton_schulz: these gradients' singular values, 0.003 to 0.2
        # of the norm, all grow to about 1 within the five steps
        assert ((O.get() - want).norm() / want.norm()).item() <= 15 ** 0.5 * 2.0 ** -11 * 2 + 2.0 ** -8 / 3 ** 0.5
