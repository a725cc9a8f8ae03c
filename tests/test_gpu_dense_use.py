"""The layer calls as programs use them: captured into graphs and replayed, on
several streams at once, repeated, next to memory that holds NaN, at the largest
arrays they take, and with arguments the binding refuses."""
import threading

import numpy as np
import pytest
import torch

import dense_gemm_14_amd as g
from tests.dense_util import Out, randn, workspace
from tests.gpu_util import need_gpu
from tests.test_gpu_dense import gen_of

pytestmark = pytest.mark.gpu


def bf(gen, *shape, std=1.0):
    return randn(gen, *shape, std=std).cuda()


class Layer:
    """A gated layer's arrays and calls, each with its own workspace."""

    def __init__(self, M, N, K, seed):
        gen = gen_of(seed, M, N, K)
        self.M, self.N, self.K = M, N, K
        self.A, self.B, self.bias = bf(gen, M, K), bf(gen, 2 * N, K, std=K ** -0.5), bf(gen, 2 * N)
        self.R, self.dC = bf(gen, M, K), bf(gen, M, N, std=2.0 ** -8)
        self.W = bf(gen, K, N, std=N ** -0.5)
        new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
        self.C, self.Z, self.Y = new(M, N), new(M, 2 * N), new(M, K)
        self.dA, self.dB, self.dbias = new(M, K), new(2 * N, K), new(2 * N)
        self.dH, self.dW, self.O = new(M, N), new(K, N), new(2 * N, K)
        nb = max(g.gated_workspace_size(M, N, K), g.gated_bwd_workspace_size(M, N, K),
                 g.bias_act_res_workspace_size(M, K, N), g.bias_act_bwd_workspace_size(M, K, N, g.ACT_GELU_TANH),
                 g.newton_schulz_workspace_size(1, 2 * N, K))
        self.ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        self.outs = (self.C, self.Z, self.Y, self.dA, self.dB, self.dbias, self.dH, self.dW, self.O)

    def run(self):
        M, N, K, ws = self.M, self.N, self.K, self.ws
        g.gemm_bf16_nt_gated(M, N, K, self.A, self.B, self.bias, g.ACT_SILU, self.Z, self.C, ws)
        g.gemm_bf16_nt_bias_act_res(M, K, N, self.C, self.W, None, g.ACT_NONE, self.R, None, self.Y, ws)
        g.gemm_bf16_nt_bias_act_bwd(M, K, N, self.C, self.W, self.Y, g.ACT_GELU_TANH, self.R, self.dH, self.dW, None, ws)
        g.gemm_bf16_nt_gated_bwd(M, N, K, self.A, self.B, self.Z, g.ACT_SILU, self.dC, self.dA, self.dB, self.dbias, ws)
        g.newton_schulz(1, 2 * N, K, self.dB, self.O, workspace=ws)

    def wipe(self):
        for o in self.outs:
            o.view(torch.int16).fill_(0x7FC1)


# sizes that take small tiles, 128 x 128 with split K, and 256 x 256 tiles
SIZES = [(5, 136, 72), (200, 264, 520), (700, 1032, 1544), (2050, 2056, 2048)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_captured_and_replayed(M, N, K):
    need_gpu()
    print("graph", M, N, K, flush=True)
    layer = Layer(M, N, K, 1)
    layer.run()
    torch.cuda.synchronize()
    want = [o.clone() for o in layer.outs]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    layer.wipe()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        layer.run()
    for r in range(3):
        layer.wipe()        # eager work between the replays
        layer.ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, w) in enumerate(zip(layer.outs, want)):
            assert torch.equal(o, w), (r, i)
    del graph


@pytest.mark.parametrize("kernel", [g.LAYER_AUTO, g.LAYER_LARGE, g.LAYER_SPLIT, g.LAYER_TILE, g.LAYER_SMALL, g.LAYER_NARROW])
def test_streams_side_by_side_and_repeated(kernel):
    # two layers on two streams of default priority, interleaved call by call;
    # every result equals the one computed alone, bit by bit
    need_gpu()
    g.force_layer_kernel(kernel)
    try:
        layers = [Layer(600, 520, 776, 3), Layer(333, 1032, 520, 4)]
        want = []
        for layer in layers:
            layer.run()
            torch.cuda.synchronize()
            want.append([o.clone() for o in layer.outs])
        streams = [torch.cuda.Stream() for _ in layers]
        for r in range(6):
            for layer in layers:
                layer.wipe()
            torch.cuda.synchronize()
            for layer, s in zip(layers, streams):
                with torch.cuda.stream(s):
                    layer.run()
            torch.cuda.synchronize()
            for k, layer in enumerate(layers):
                for i, (o, w) in enumerate(zip(layer.outs, want[k])):
                    assert torch.equal(o, w), (kernel, r, k, i)
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)


def test_threads_with_a_stream_each():
    # calls from several threads at once, while another thread changes the
    # kernels' override: a call runs as planned or is refused for its workspace
    need_gpu()
    layers = [Layer(130 + 40 * i, 264, 520, 80 + i) for i in range(4)]
    want = []
    for layer in layers:
        layer.run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in layer.outs])
    refused = [0] * len(layers)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                try:
                    layers[i].run()
                except g.Gemm355Error as e:
                    assert e.status == g.ERR_UNSUPPORTED
                    refused[i] += 1
            torch.cuda.current_stream().synchronize()

    def toggle():
        for k in [g.LAYER_SPLIT, g.LAYER_TILE, g.LAYER_SMALL, g.LAYER_AUTO] * 25:
            g.force_layer_kernel(k)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(layers))] + [threading.Thread(target=toggle)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    g.force_layer_kernel(g.LAYER_AUTO)
    torch.cuda.synchronize()
    for layer, w in zip(layers, want):
        layer.wipe()
        layer.run()
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(layer.outs, w))


@pytest.mark.parametrize("kernel", [g.LAYER_LARGE, g.LAYER_SPLIT, g.LAYER_TILE, g.LAYER_SMALL, g.LAYER_NARROW])
@pytest.mark.parametrize("M,N,K", [(77, 136, 264), (301, 520, 328)])
def test_memory_around_the_inputs_does_not_matter(kernel, M, N, K):
    # every input between bands of NaN: the results are those of inputs alone
    need_gpu()
    gen = gen_of(51, M, N, K)
    A, B, bias, R = randn(gen, M, K), randn(gen, 2 * N, K), randn(gen, 2 * N), randn(gen, M, N)
    Z, dC = randn(gen, M, 2 * N), randn(gen, M, N)
    G = randn(gen, 3, N, K)

    def run(wrap):
        a, b, bi, r, z, dc, gg = (wrap(x) for x in (A, B, bias, R, Z, dC, G))
        C, C2, dA, dB, db, O = Out(M, N), Out(M, N), Out(M, K), Out(2 * N, K), Out(2 * N), Out(3, N, K)
        nb = max(g.gated_workspace_size(M, N, K), g.gated_bwd_workspace_size(M, N, K),
                 g.bias_act_res_workspace_size(M, N, K), g.newton_schulz_workspace_size(3, N, K))
        ws, nb, check = workspace(nb)
        g.gemm_bf16_nt_gated(M, N, K, a, b, bi, g.ACT_SILU, None, C.t, ws, nb)
        g.gemm_bf16_nt_bias_act_res(M, N, K, a, b[:N], bi[:N], g.ACT_RELU, r, None, C2.t, ws, nb)
        g.gemm_bf16_nt_gated_bwd(M, N, K, a, b, z, g.ACT_SILU, dc, dA.t, dB.t, db.t, ws, nb)
        g.newton_schulz(3, N, K, gg, O.t, workspace=ws, workspace_bytes=nb)
        torch.cuda.synchronize()
        check()
        return [x.get() for x in (C, C2, dA, dB, db, O)]
    g.force_layer_kernel(kernel)
    try:
        plain = run(lambda x: x.cuda())
        banded = run(lambda x: Out(*x.shape, fill=x.cuda()).t)
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)
    for i, (p, b) in enumerate(zip(plain, banded)):
        assert torch.isfinite(b).all() and torch.equal(p, b), i


@pytest.mark.parametrize("kernel", [g.LAYER_AUTO, g.LAYER_LARGE, g.LAYER_TILE, g.LAYER_SMALL])
def test_largest_arrays(kernel):
    # Z and dZ of 2.139e9 bytes, just inside the limit of 2^31: offsets with
    # the top bit set below it. Whole numbers: exact sums, sampled rows.
    need_gpu()
    M, N, K = 65280, 8192, 256
    gen = torch.Generator(device="cuda")
    gen.manual_seed(61)
    whole = lambda top, *s: torch.randint(-top, top + 1, s, generator=gen, device="cuda").to(torch.bfloat16)
    A, B = whole(1, M, K), whole(1, 2 * N, K)
    C, Z = (torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (N, 2 * N))
    g.force_layer_kernel(kernel)
    try:
        ws = torch.empty(max(g.gated_workspace_size(M, N, K), g.gated_bwd_workspace_size(M, N, K), 16), dtype=torch.uint8,
                         device="cuda")
        print("largest", kernel, ws.numel(), flush=True)
        g.gemm_bf16_nt_gated(M, N, K, A, B, None, g.ACT_RELU, Z, C, ws)
        torch.cuda.synchronize()
        rows = torch.tensor([0, 1, 255, 256, 31999, 32767, 32768, 65023, 65024, 65278, 65279], device="cuda")
        z = A[rows].float() @ B.float().t()
        assert torch.equal(Z[rows], z.bfloat16())
        assert torch.equal(C[rows], (z[:, :N].clamp(min=0) * z[:, N:]).bfloat16())
        # gradients: dC is zero but in a few rows and columns of 1, so that
        # every sum stays exact
        dC = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        dC[rows] = 1
        Z.fill_(1.0)
        dA, dB, db = (torch.empty(*s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (2 * N, K), (2 * N,)))
        g.gemm_bf16_nt_gated_bwd(M, N, K, A, B, Z, g.ACT_RELU, dC, dA, dB, db, ws)
        torch.cuda.synchronize()
        assert torch.equal(dA[rows], B.float().sum(0).expand(len(rows), K).bfloat16())
        other = torch.ones(M, dtype=torch.bool, device="cuda")
        other[rows] = False
        assert not dA[other].any()
        assert torch.equal(dB, A[rows].float().sum(0).expand(2 * N, K).bfloat16())
        assert torch.equal(db, torch.full_like(db, float(len(rows))))
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)


def test_newton_schulz_follows_its_rounding():
    # the same steps in 64 bits with a rounding to FP16 where the kernels round:
    # what is left is FP32 sums that fall on the other side of a rounding
    need_gpu()
    a, b, c = 3.4445, -4.7750, 2.0315
    for rows, cols in ((64, 200), (392, 264), (1032, 256)):
        gen = gen_of(71, rows, cols)
        G = randn(gen, 1, rows, cols)
        O = Out(1, rows, cols)
        ws, nb, check = workspace(g.newton_schulz_workspace_size(1, rows, cols))
        g.newton_schulz(1, rows, cols, G.cuda(), O.t, workspace=ws, workspace_bytes=nb)
        torch.cuda.synchronize()
        check()
        h = lambda t: t.half().double()
        x = G[0].double() if rows <= cols else G[0].double().t()
        scale = 2.0 ** np.ceil(0.5 * np.log2(min(rows, cols)))
        x = h(x / (x.norm() + 1e-7) * scale)
        for i in range(5):
            s = h(x @ x.t() * 256 / scale ** 2)
            p = h(a * 256 * torch.eye(len(s)).double() + b * s + c / 256 * (s @ s))
            x = p @ x / 256
            x = h(x) if i < 4 else x / scale
        want = (x if rows <= cols else x.t()).bfloat16().double()
        rel = ((O.get()[0] - want).norm() / want.norm()).item()
        # one value in forty on the other side of a BF16 border (2^-8 of it):
        # 2^-8 / sqrt(40) = 6e-4; three times that
        assert rel <= 2e-3, (rows, cols, rel)


def test_binding_refuses():
    need_gpu()
    M, N, K = 16, 64, 64
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    A, B, C = t(M, K), t(N, K), t(M, N)
    with pytest.raises(ValueError, match="device 0"):
        g._addr(A, 0, "A", 1)
    with pytest.raises(ValueError, match="must be on the GPU"):
        g.gemm_bf16_nt_bias_act_res(M, N, K, A.cpu(), B, None, 0, None, None, C)
    with pytest.raises(ValueError, match="contiguous"):
        g.gemm_bf16_nt_gated(M, N // 2, K, A.t(), B, None, 0, None, C)
    with pytest.raises(ValueError, match="holds"):
        g.gemm_bf16_nt_gated(M, N, K, A, B, None, 0, None, C)          # B has N rows, not 2 N
    with pytest.raises(ValueError, match="holds"):
        g.gemm_bf16_nt_bias_act_bwd(M, N, K, A, B, None, 0, C, A, B, t(N - 8))
    with pytest.raises(TypeError):
        g.gemm_bf16_nt_bias_act_res(M, N, K, "A", B, None, 0, None, None, C)
    with pytest.raises(TypeError):
        g.newton_schulz(1, 64, 64, A.double(), C)
    with pytest.raises(g.Gemm355Error) as e:
        g.newton_schulz(1, 64, 64, B, t(64, 64))       # no workspace
    assert e.value.status == g.ERR_INVALID_ARG
    with pytest.raises(g.Gemm355Error) as e:
        g.newton_schulz(1, 64, 64, B, t(64, 64), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == g.ERR_UNSUPPORTED


def test_binding_takes_every_kind_of_argument():
    # tensors, parameters, raw addresses, numpy sizes, streams as objects and as
    # addresses, a workspace with its size: the same results
    need_gpu()
    M, N, K = 40, 136, 4104
    gen = gen_of(91)
    A, B, R = bf(gen, M, K), bf(gen, N, K, std=K ** -0.5), bf(gen, M, N)
    nb = max(g.bias_act_res_workspace_size(M, N, K), g.bias_act_bwd_workspace_size(M, N, K, g.ACT_SILU))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    results = []
    param = torch.nn.Parameter(B)
    for sizes, arg, w, stream in (((M, N, K), lambda t: t, (ws,), None),
                                  (np.array([M, N, K]), lambda t: t.data_ptr(), (ws.data_ptr(), nb), s.cuda_stream),
                                  ((M, N, K), lambda t: param if t is B else t, (ws, nb), s)):
        C, Z, dA, dB, db = new(M, N), new(M, N), new(M, K), new(N, K), new(N)
        g.gemm_bf16_nt_bias_act_res(*sizes, arg(A), arg(B), None, g.ACT_SILU, arg(R), arg(Z), arg(C), *w, stream=stream)
        g.gemm_bf16_nt_bias_act_bwd(*sizes, arg(A), arg(B), arg(Z), g.ACT_SILU, arg(R), arg(dA), arg(dB), arg(db), *w,
                                    stream=stream)
        torch.cuda.synchronize()
        results.append((C, Z, dA, dB, db))
    for r in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, results[0]))
    C = new(M, N)
    with pytest.raises(ValueError, match="workspace_bytes"):
        g.gemm_bf16_nt_bias_act_res(M, N, K, A, B, None, 0, None, None, C, ws.data_ptr())
    with pytest.raises(ValueError, match="workspace"):
        g.gemm_bf16_nt_bias_act_res(M, N, K, A, B, None, 0, None, None, C, ws, nb + 1)
    with pytest.raises(ValueError, match="GPU"):
        g.gemm_bf16_nt_bias_act_res(M, N, K, A, B, None, 0, None, None, C, ws.cpu())
    with pytest.raises(OverflowError):
        g.gemm_bf16_nt_bias_act_res(1 << 40, N, K, A, B, None, 0, None, None, C, ws)
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm_bf16_nt_bias_act_res(-M, N, K, A, B, None, 0, None, None, C, ws)
    assert e.value.status == g.ERR_INVALID_ARG
    # what was refused left nothing behind: the next call is right
    g.gemm_bf16_nt_bias_act_res(M, N, K, A, B, None, g.ACT_SILU, R, None, C, ws)
    torch.cuda.synchronize()
    assert torch.equal(C, results[0][0])
