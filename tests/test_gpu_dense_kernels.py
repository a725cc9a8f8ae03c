"""Every kernel of the layer calls' products, forced in turn: whole and split
256 x 256 tiles and 128 x 128 tiles give the right values at sizes that cross
their borders, in every layout, with one tile and with several rounds of them."""
import pytest
import torch

import dense_gemm_14_amd as g
from tests.dense_util import Out, backward, close, forward, randn, workspace
from tests.gpu_util import need_gpu
from tests.test_gpu_dense import dev, gen_of, ortho_exact, run_backward, run_forward, run_ortho

pytestmark = pytest.mark.gpu
KERNELS = [g.LAYER_LARGE, g.LAYER_SPLIT, g.LAYER_TILE, g.LAYER_SMALL, g.LAYER_NARROW]


@pytest.fixture(params=KERNELS, ids=["large", "split", "tile", "small", "narrow"])
def kernel(request):
    need_gpu()
    g.force_layer_kernel(request.param)
    yield request.param
    g.force_layer_kernel(g.LAYER_AUTO)


@pytest.mark.parametrize("M,N,K", [(8, 8, 256), (300, 264, 520), (257, 520, 1032), (513, 1032, 200)])
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_layers(kernel, gated, M, N, K):
    rows = 2 * N if gated else N
    gen = gen_of(M, N, K, 31)
    A, B, bias = randn(gen, M, K), randn(gen, rows, K, std=K ** -0.5), randn(gen, rows)
    R = None if gated else randn(gen, M, N)
    print("kernel", kernel, gated, M, N, K, flush=True)
    C, Z = run_forward(gated, M, N, K, A, B, bias, g.ACT_GELU_TANH, R, True)
    y, ey, z, ez = forward(A, B, bias, g.ACT_GELU_TANH, R, gated)
    close(C, y, ey, "C")
    close(Z, z, ez, "Z")
    dC, Zin = randn(gen, M, N), randn(gen, M, rows)
    got = run_backward(gated, M, N, K, A, B, Zin, g.ACT_SILU, dC)
    for k, (v, e) in backward(A, B, Zin, g.ACT_SILU, dC, gated).items():
        close(got[k], v, e, k)


@pytest.mark.parametrize("shape", [(1, 520, 264), (2, 264, 776), (1, 1032, 1032), (3, 776, 520)])
def test_newton_schulz(kernel, shape):
    gen = gen_of(*shape, 37)
    G = (torch.randn(*shape, generator=gen) * 1e-3)
    print("kernel", kernel, shape, flush=True)
    got, want = run_ortho(G), ortho_exact(G, 5, (3.4445, -4.7750, 2.0315), 1e-7)
    rel = ((got - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max().item()
    assert rel <= 15 ** 0.5 * 2.0 ** -11 * 2 + 2.0 ** -8 / 3 ** 0.5, rel


@pytest.mark.parametrize("batch,side", [(20, 784), (5, 1160)], ids=["256-tiles", "192-tiles"])
def test_newton_schulz_whole_symmetric_tiles(batch, side):
    # whole 256 x 256 tiles where 192 x 192 ones need another round, and those
    # over more than one round's and with ragged edges
    need_gpu()
    gen = gen_of(batch, side, 39)
    G = torch.randn(batch, side, side, generator=gen)
    g.force_layer_kernel(g.LAYER_LARGE)
    try:
        print("newton schulz", batch, side, flush=True)
        got = run_ortho(G, 2)
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)
    want = ortho_exact(G.cuda(), 2, (3.4445, -4.7750, 2.0315), 1e-7).cpu()
    rel = ((got - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max().item()
    assert rel <= 6 ** 0.5 * 2.0 ** -11 * 2 + 2.0 ** -8 / 3 ** 0.5, rel


def whole(gen, *shape, top=2):
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [(4608, 4600, 328), (6200, 6152, 256), (1032, 2056, 4104)])
def test_many_tiles_are_exact(kernel, M, N, K):
    # whole numbers whose sums are exact in FP32: one right value each; more
    # tiles than workgroups, so items follow each other in one workgroup
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    A, B, R, dC = whole(gen, M, K), whole(gen, N, K), whole(gen, M, N), whole(gen, M, N, top=1)
    print("kernel", kernel, M, N, K, flush=True)
    C, dA, dB, dbias = Out(M, N), Out(M, K), Out(N, K), Out(N)
    ws, nb, check = workspace(max(g.bias_act_res_workspace_size(M, N, K),
                                  g.bias_act_bwd_workspace_size(M, N, K, g.ACT_NONE)))
    for _ in range(2):     # twice: nothing is left behind in the workspace
        g.gemm_bf16_nt_bias_act_res(M, N, K, A, B, None, g.ACT_RELU, R, None, C.t, ws, nb)
        g.gemm_bf16_nt_bias_act_bwd(M, N, K, A, B, None, g.ACT_NONE, dC, dA.t, dB.t, dbias.t, ws, nb)
        torch.cuda.synchronize()
        check()
        a, b, d = A.float(), B.float(), dC.float()
        for got, want in ((C, ((a @ b.t()).clamp(min=0) + R.float())), (dA, d @ b), (dB, d.t().contiguous() @ a),
                          (dbias, d.sum(0))):
            assert torch.equal(got.get(), want.bfloat16().double().cpu())


@pytest.mark.parametrize("choice", [g.LAYER_AUTO, g.LAYER_SMALL], ids=["auto", "small"])
@pytest.mark.parametrize("M,N,K", [(1100, 1104, 1104), (64, 18000, 520), (2001, 664, 104), (170, 1528, 1608),
                                   (1310, 6288, 168), (4100, 4104, 72)])
def test_small_tiles_around_one_per_unit_are_exact(choice, M, N, K):
    # between one and two 64 x 64 tiles per compute unit, in one product or in
    # both of a backward pass: workgroups of four waves, two to a unit; the last
    # two, about eight and sixteen of a short contraction: of one
    need_gpu()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    A, B, dC = whole(gen, M, K), whole(gen, N, K), whole(gen, M, N, top=1)
    print("choice", choice, M, N, K, flush=True)
    C, dA, dB, dbias = Out(M, N), Out(M, K), Out(N, K), Out(N)
    g.force_layer_kernel(choice)
    try:
        ws, nb, check = workspace(max(g.bias_act_res_workspace_size(M, N, K),
                                      g.bias_act_bwd_workspace_size(M, N, K, g.ACT_NONE)))
        g.gemm_bf16_nt_bias_act_res(M, N, K, A, B, None, g.ACT_NONE, None, None, C.t, ws, nb)
        g.gemm_bf16_nt_bias_act_bwd(M, N, K, A, B, None, g.ACT_NONE, dC, dA.t, dB.t, dbias.t, ws, nb)
        torch.cuda.synchronize()
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)
    check()
    a, b, d = A.float(), B.float(), dC.float()
    for got, want in ((C, a @ b.t()), (dA, d @ b), (dB, d.t().contiguous() @ a), (dbias, d.sum(0))):
        assert torch.equal(got.get(), want.bfloat16().double().cpu())


def test_kernels_agree_with_the_workspace_each_asks_for():
    need_gpu()
    M, N, K = 700, 1032, 520
    gen = gen_of(41)
    A, B = randn(gen, M, K), randn(gen, N, K)
    try:
        for k in KERNELS + [g.LAYER_AUTO]:
            g.force_layer_kernel(k)
            nb = g.bias_act_res_workspace_size(M, N, K)
            if nb:
                ws, _, _ = workspace(nb)
                with pytest.raises(g.Gemm355Error) as e:
                    g.gemm_bf16_nt_bias_act_res(M, N, K, dev(A), dev(B), None, 0, None, None, Out(M, N).t, ws, nb - 1)
                assert e.value.status == g.ERR_UNSUPPORTED
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)
