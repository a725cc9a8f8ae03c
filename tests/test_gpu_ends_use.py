"""Embedding, layer norm and cross entropy as programs use them: a whole training
step together with the layers between them, against the same steps in 64 bits;
captured into a graph and replayed; on several streams and threads at once; next to
memory that holds NaN; with every kind of argument the binding takes, and those it
refuses."""
import threading

import numpy as np
import pytest
import torch

import dense_gemm_14_amd as g
from tests.gpu_util import need_gpu
from tests.rows_util import Array, randn

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
EPS, SCALE = 1e-5, 8.0


def gen_of(seed):
    gen = torch.Generator()
    gen.manual_seed(seed)
    return gen


class Step:
    """One training step of a network of one gated block: token ids in, the rows'
    losses and every gradient out. The table is the output projection, too."""

    def __init__(self, T, V, K, N, seed, stream=BF16):
        gen = gen_of(seed)
        self.T, self.V, self.K, self.N, self.stream = T, V, K, N, stream
        put = lambda x: x.cuda()
        self.ids = put(torch.randint(0, V, (T,), generator=gen))
        targets = torch.randint(0, V, (T,), generator=gen)
        targets[torch.rand(T, generator=gen) < 0.2] = -100
        self.targets = put(targets.int())
        self.E = put(randn(gen, V, K, std=K ** -0.5))
        self.W1, self.W2 = put(randn(gen, 2 * N, K, std=K ** -0.5)), put(randn(gen, K, N, std=N ** -0.5))
        self.g1, self.b1 = put(1 + randn(gen, K, std=0.2)), put(randn(gen, K, std=0.2))
        self.g2, self.b2 = put(1 + randn(gen, K, std=0.2)), put(randn(gen, K, std=0.2))
        kept = (self.targets >= 0)
        self.dloss = (kept.float() / kept.sum().clamp(min=1)).contiguous()
        new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")
        self.x0, self.y1, self.c, self.z, self.x1, self.y2 = new(T, K), new(T, K), new(T, N), new(T, 2 * N), new(T, K), new(T, K)
        self.m1, self.r1, self.m2, self.r2, self.loss, self.lse = (new(T, dtype=FP32) for _ in range(6))
        self.dy2, self.dx1, self.dc, self.dy1, self.dx0 = new(T, K), new(T, K), new(T, N), new(T, K), new(T, K)
        self.dE, self.dW1, self.dW2 = new(V, K), new(2 * N, K), new(K, N)
        self.dg1, self.db1, self.dg2, self.db2 = (new(K) for _ in range(4))
        nb = max(g.gated_workspace_size(T, N, K), g.bias_act_res_workspace_size(T, K, N), g.cross_entropy_workspace_size(T, V, K),
                 g.cross_entropy_bwd_workspace_size(T, V, K), g.layer_norm_bwd_workspace_size(T, K),
                 g.bias_act_bwd_workspace_size(T, K, N, g.ACT_NONE), g.gated_bwd_workspace_size(T, N, K),
                 g.embedding_bwd_workspace_size(T, V, K))
        self.ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        self.outs = (self.loss, self.lse, self.y2, self.dE, self.dW1, self.dW2, self.dg1, self.db1, self.dg2, self.db2, self.dx0)

    def run(self):
        T, V, K, N, ws = self.T, self.V, self.K, self.N, self.ws
        g.embedding(T, V, K, self.ids, self.E, self.x0, SCALE)
        g.layer_norm(T, K, self.x0, self.g1, self.b1, self.y1, self.m1, self.r1, EPS)
        g.gemm_bf16_nt_gated(T, N, K, self.y1, self.W1, None, g.ACT_SILU, self.z, self.c, ws)
        g.gemm_bf16_nt_bias_act_res(T, K, N, self.c, self.W2, None, g.ACT_NONE, self.x0, None, self.x1, ws)
        g.layer_norm(T, K, self.x1, self.g2, self.b2, self.y2, self.m2, self.r2, EPS)
        g.gemm_bf16_nt_cross_entropy(T, V, K, self.y2, self.E, self.targets, self.loss, self.lse, ws)
        g.gemm_bf16_nt_cross_entropy_bwd(T, V, K, self.y2, self.E, self.targets, self.lse, self.dloss, self.dy2, self.dE, ws)
        g.layer_norm_bwd(T, K, self.x1, self.g2, self.m2, self.r2, self.dy2, None, self.dx1, self.dg2, self.db2, ws)
        g.gemm_bf16_nt_bias_act_bwd(T, K, N, self.c, self.W2, None, g.ACT_NONE, self.dx1, self.dc, self.dW2, None, ws)
        g.gemm_bf16_nt_gated_bwd(T, N, K, self.y1, self.W1, self.z, g.ACT_SILU, self.dc, self.dy1, self.dW1, None, ws)
        g.layer_norm_bwd(T, K, self.x0, self.g1, self.m1, self.r1, self.dy1, self.dx1, self.dx0, self.dg1, self.db1, ws)
        g.embedding_bwd(T, V, K, self.ids, self.dx0, self.dE, self.dE, SCALE, ws)

    def wipe(self):
        for o in self.outs:
            o.fill_(float("nan"))


def rounded_reference(s):
    """The step in 64 bits with a rounding to BF16 where the calls round."""
    q = lambda t: t.bfloat16().double()
    E, W1, W2, g1, b1, g2, b2 = (x.cpu().double() for x in (s.E, s.W1, s.W2, s.g1, s.b1, s.g2, s.b2))
    ids, t, w, N, K = s.ids.cpu(), s.targets.cpu().long(), s.dloss.cpu().double()[:, None], s.N, s.K

    def norm(x, ga, be):
        m, v = x.mean(1, keepdim=True), x.var(1, correction=0, keepdim=True)
        r = 1 / torch.sqrt(v + EPS)
        return q((x - m) * r * ga + be), (x - m) * r, r

    def norm_bwd(u, r, ga, dy, extra):
        h = dy * ga
        return q(r * (h - h.mean(1, keepdim=True) - u * (h * u).mean(1, keepdim=True)) + extra), q((dy * u).sum(0)), q(dy.sum(0))
    x0 = q(SCALE * E[ids])
    y1, u1, r1 = norm(x0, g1, b1)
    z = y1 @ W1.t()
    c = q(torch.nn.functional.silu(z[:, :N]) * z[:, N:])
    z = q(z)
    x1 = q(c @ W2.t() + x0)
    y2, u2, r2 = norm(x1, g2, b2)
    logits = y2 @ E.t()
    lse = torch.logsumexp(logits, 1, keepdim=True)
    kept, at = (t >= 0)[:, None], t.clamp(min=0)[:, None]
    loss = torch.where(kept, lse - logits.gather(1, at), 0.0)
    dz = torch.exp(logits - lse)
    dz.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    dz = q(torch.where(kept, dz * (w / w.max()), 0.0))
    dy2, dE = q(dz @ E * w.max()), q(dz.t() @ y2 * w.max())
    dx1, dg2, db2 = norm_bwd(u2, r2, g2, dy2, 0.0)
    dc, dW2 = q(dx1 @ W2), q(dx1.t() @ c)
    a, b = z[:, :N], z[:, N:]
    sg = torch.sigmoid(a)
    dh = q(torch.cat([dc * b * (sg + a * sg * (1 - sg)), dc * a * sg], 1))
    dy1, dW1 = q(dh @ W1), q(dh.t() @ y1)
    dx0, dg1, db1 = norm_bwd(u1, r1, g1, dy1, dx1)
    dE = q(dE + SCALE * torch.zeros_like(dE).index_add_(0, ids, dx0))
    return dict(loss=loss[:, 0], y2=y2, dE=dE, dW1=dW1, dW2=dW2, dg1=dg1, db1=db1, dg2=dg2, db2=db2, dx0=dx0)


SIZES = [(200, 515, 136, 264), (900, 1031, 264, 520), (1, 77, 72, 136), (1500, 300, 72, 72)]


@pytest.mark.parametrize("T,V,K,N", SIZES)
def test_a_training_step(T, V, K, N):
    need_gpu()
    print("step", T, V, K, N, flush=True)
    s = Step(T, V, K, N, 1)
    if T == 1:
        s.targets.fill_(5)
        s.dloss.fill_(1.0)
    s.wipe()
    s.run()
    torch.cuda.synchronize()
    want = rounded_reference(s)
    for k, w in want.items():
        got = getattr(s, k).cpu().double()
        # What is left are values on the other side of a rounding, one step of BF16
        # (2^-7 of the value) each: sums in FP32 move one value in a hundred across,
        # and each of the up to twelve roundings in a row passes on what the ones
        # before it did. 12 sqrt(2^-14 / 100) = 9e-3 if all add up in the same
        # direction.
        rel = ((got - w).norm() / w.norm().clamp(min=1e-30)).item()
        assert rel <= 9e-3, (k, rel)
    # the gradients are those of the mean loss: against autograd in 64 bits, with up to
    # twelve roundings of 2^-8 between the two
    E, W1, W2, g1, b1, g2, b2 = leaves = [x.cpu().double().requires_grad_() for x in
                                          (s.E, s.W1, s.W2, s.g1, s.b1, s.g2, s.b2)]
    F = torch.nn.functional
    x0 = SCALE * E[s.ids.cpu()]
    z = F.layer_norm(x0, (K,), g1, b1, EPS) @ W1.t()
    x1 = (F.silu(z[:, :N]) * z[:, N:]) @ W2.t() + x0
    logits = F.layer_norm(x1, (K,), g2, b2, EPS) @ E.t()
    F.cross_entropy(logits, s.targets.cpu().long()).backward()
    for k, leaf in zip(("dE", "dW1", "dW2", "dg1", "db1", "dg2", "db2"), leaves):
        rel = ((getattr(s, k).cpu().double() - leaf.grad).norm() / leaf.grad.norm().clamp(min=1e-30)).item()
        assert rel <= 12 * 2.0 ** -8, (k, rel)


@pytest.mark.parametrize("T,V,K,N", SIZES + [(2100, 9000, 264, 264), (99000, 3001, 64, 72)])
def test_captured_and_replayed(T, V, K, N):
    need_gpu()
    print("graph", T, V, K, N, flush=True)
    s = Step(T, V, K, N, 2)
    s.run()
    torch.cuda.synchronize()
    want = [o.clone() for o in s.outs]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wipe()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        s.run()
    for r in range(3):
        s.wipe()        # eager work between the replays
        s.ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, w) in enumerate(zip(s.outs, want)):
            assert torch.equal(o, w), (r, i)
    # other ids and targets in the same arrays: a replay reads them anew
    s.ids.copy_(torch.randint(0, V, (T,), generator=gen_of(3)))
    s.targets.copy_(torch.randint(-1, V, (T,), generator=gen_of(4)).int())
    s.run()
    torch.cuda.synchronize()
    want = [o.clone() for o in s.outs]
    s.wipe()
    graph.replay()
    torch.cuda.synchronize()
    for i, (o, w) in enumerate(zip(s.outs, want)):
        assert torch.equal(o, w), i
    del graph


def test_streams_side_by_side():
    need_gpu()
    steps = [Step(1100, 700, 264, 136, 5), Step(300, 2000, 136, 264, 6)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in s.outs])
    streams = [torch.cuda.Stream() for _ in steps]
    for r in range(6):
        for s in steps:
            s.wipe()
        torch.cuda.synchronize()
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
        torch.cuda.synchronize()
        for k, s in enumerate(steps):
            for i, (o, w) in enumerate(zip(s.outs, want[k])):
                assert torch.equal(o, w), (r, k, i)


def test_threads_with_a_stream_each():
    need_gpu()
    steps = [Step(130 + 300 * i, 400, 136, 136, 20 + i) for i in range(4)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in s.outs])
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for r in range(8):
                steps[i].wipe()
                steps[i].run()
                torch.cuda.current_stream().synchronize()
                wrong.extend((i, r, k) for k, (o, w) in enumerate(zip(steps[i].outs, want[i])) if not torch.equal(o, w))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(steps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def banded(x):
    """x between two bands of NaN (ids: of ids far outside)."""
    if x.is_floating_point():
        return Array(*x.shape, dtype=x.dtype, fill=x.cuda()).t
    buf = torch.full((x.numel() + 1024,), 1 << 30, dtype=x.dtype, device="cuda")
    buf[512:512 + x.numel()] = x.cuda()
    return buf[512:512 + x.numel()]


@pytest.mark.parametrize("kernel", [g.LAYER_AUTO, g.LAYER_LARGE, g.LAYER_SPLIT, g.LAYER_TILE, g.LAYER_SMALL, g.LAYER_NARROW])
@pytest.mark.parametrize("M,V,K", [(77, 137, 264), (301, 523, 328)])
def test_memory_around_the_arrays_does_not_matter(M, V, K, kernel):
    need_gpu()
    gen = gen_of(51)
    A, B, X = randn(gen, M, K), randn(gen, V, K, std=K ** -0.5), randn(gen, M, K, dtype=FP32)
    t = torch.randint(-1, V, (M,), generator=gen)
    ga, lse, w = randn(gen, K, dtype=FP32), torch.randn(M, generator=gen) + 8, torch.randn(M, generator=gen)
    mean, rstd = torch.randn(M, generator=gen), torch.rand(M, generator=gen) + 0.5

    def run(wrap):
        a, b, x, ids, gamma, l, wt, m, r = (wrap(v) for v in (A, B, X, t, ga, lse, w, mean, rstd))
        outs = [Array(M, dtype=FP32), Array(M, dtype=FP32), Array(M, K), Array(V, K), Array(M, K), Array(M, K, dtype=FP32),
                Array(K, dtype=FP32), Array(K, dtype=FP32), Array(M, K, dtype=FP32), Array(V, K, dtype=FP32)]
        o = [x.t for x in outs]
        nb = max(g.cross_entropy_workspace_size(M, V, K), g.cross_entropy_bwd_workspace_size(M, V, K),
                 g.layer_norm_bwd_workspace_size(M, K), g.embedding_bwd_workspace_size(M, V, K))
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
        g.gemm_bf16_nt_cross_entropy(M, V, K, a, b, ids, o[0], o[1], ws)
        g.gemm_bf16_nt_cross_entropy_bwd(M, V, K, a, b, ids, l, wt, o[2], o[3], ws)
        g.layer_norm(M, K, x, gamma, None, o[4], None, None)
        g.layer_norm_bwd(M, K, x, gamma, m, r, a, None, o[5], o[6], o[7], ws)
        g.embedding(M, V, K, ids, b, o[8])
        g.embedding_bwd(M, V, K, ids, a, None, o[9], 1.0, ws)
        torch.cuda.synchronize()
        return [x.get() for x in outs]
    g.force_layer_kernel(kernel)
    try:
        plain, between = run(lambda v: v.cuda()), run(banded)
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)
    for i, (p, b) in enumerate(zip(plain, between)):
        assert torch.isfinite(b).all() and torch.equal(p, b), i


def test_numbers_per_row_may_lie_anywhere():
    # ids and FP32 values per row at addresses that only their own type aligns
    need_gpu()
    M, V, K = 301, 300, 72
    gen = gen_of(61)
    A, B = randn(gen, M, K).cuda(), randn(gen, V, K).cuda()
    for it in (torch.int32, torch.int64):
        t = torch.randint(-1, V, (M + 1,), generator=gen).to(it).cuda()
        f = [torch.empty(M + 1, device="cuda") for _ in range(4)]
        ws = torch.empty(max(g.cross_entropy_workspace_size(M, V, K), g.cross_entropy_bwd_workspace_size(M, V, K)),
                         dtype=torch.uint8, device="cuda")
        results = []
        for ids, (loss, lse, mean, rstd) in ((t[1:], [x[1:] for x in f]), (t[1:].clone(), [x[:M].clone() for x in f])):
            dA, dB, Y, dX = torch.empty_like(A), torch.empty_like(B), torch.empty_like(A), torch.empty_like(A)
            g.gemm_bf16_nt_cross_entropy(M, V, K, A, B, ids, loss, lse, ws)
            g.gemm_bf16_nt_cross_entropy_bwd(M, V, K, A, B, ids, lse, loss, dA, dB, ws)
            g.layer_norm(M, K, A, None, None, Y, mean, rstd)
            g.layer_norm_bwd(M, K, A, None, mean, rstd, Y, None, dX, None, None)
            torch.cuda.synchronize()
            results.append([x.clone() for x in (loss, lse, mean, rstd, dA, dB, Y, dX)])
        assert all(torch.equal(x, y) for x, y in zip(*results))


def test_binding_takes_every_kind_of_argument():
    # tensors, parameters, raw addresses, bits, numpy sizes, streams as objects and as
    # addresses: the same results
    need_gpu()
    M, V, K = 1100, 300, 72
    gen = gen_of(71)
    A, E = randn(gen, M, K).cuda(), randn(gen, V, K).cuda()
    X, ga = randn(gen, M, K, dtype=FP32).cuda(), randn(gen, K, dtype=FP32).cuda()
    t = torch.randint(-1, V, (M,), generator=gen).cuda()
    nb = max(g.cross_entropy_workspace_size(M, V, K), g.cross_entropy_bwd_workspace_size(M, V, K),
             g.layer_norm_bwd_workspace_size(M, K), g.embedding_bwd_workspace_size(M, V, K))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    param = torch.nn.Parameter
    address = lambda x: x.data_ptr()
    bits = lambda x: x.view(torch.int16) if x.dtype == BF16 else x
    raw = dict(id_type=g.INT64, e_type=g.BF16, y_type=g.BF16), dict(x_type=g.FP32, w_type=g.FP32), dict(target_type=g.INT64)
    none = ({}, {}, {})
    results = []
    for sizes, arg, w, stream, types in (((M, V, K), lambda x: x, (ws,), None, none),
                                         ((M, V, K), lambda x: param(x) if x is E or x is ga else x, (ws, nb), s, none),
                                         ((M, V, K), bits, (ws,), None, none),
                                         (np.array([M, V, K]), address, (ws.data_ptr(), nb), s.cuda_stream, raw)):
        m, v, k = sizes
        new = lambda *shape, dtype=BF16: torch.empty(*shape, dtype=dtype, device="cuda")
        loss, lse, mean, rstd = (new(M, dtype=FP32) for _ in range(4))
        dA, dE, Y, Z, dX, dg, db, dT = new(M, K), new(V, K), new(M, K), new(M, K), new(M, K, dtype=FP32), \
            new(K, dtype=FP32), new(K, dtype=FP32), new(V, K)
        torch.cuda.synchronize()
        g.embedding(m, v, k, arg(t), arg(E), arg(Z), 2.0, stream=stream, **types[0])
        g.embedding_bwd(m, v, k, arg(t), arg(A), None, arg(dT), 2.0, *w, stream=stream, **types[0])
        g.layer_norm(m, k, arg(X), arg(ga), arg(ga), arg(Y), arg(mean), arg(rstd), stream=stream, **types[1])
        g.layer_norm_bwd(m, k, arg(X), arg(ga), arg(mean), arg(rstd), arg(A), None, arg(dX), arg(dg), arg(db), *w,
                         stream=stream, **types[1])
        g.gemm_bf16_nt_cross_entropy(m, v, k, arg(A), arg(E), arg(t), arg(loss), arg(lse), *w, stream=stream, **types[2])
        g.gemm_bf16_nt_cross_entropy_bwd(m, v, k, arg(A), arg(E), arg(t), arg(lse), None, arg(dA), arg(dE), *w,
                                         stream=stream, **types[2])
        torch.cuda.synchronize()
        results.append((loss, lse, mean, rstd, dA, dE, Y, Z, dX, dg, db, dT))
    for i, r in enumerate(results[1:]):
        for k, (x, y) in enumerate(zip(r, results[0])):
            assert torch.equal(x, y), (i, k)


def test_binding_refuses():
    need_gpu()
    M, V, K = 16, 40, 64
    bf = lambda *s: torch.zeros(*s, dtype=BF16, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")
    t = torch.zeros(M, dtype=torch.int64, device="cuda")
    A, B, ws = bf(M, K), bf(V, K), torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="holds"):
        g.embedding(M, V + 1, K, t, B, A)
    with pytest.raises(ValueError, match="holds"):
        g.embedding(M + 1, V, K, t, B, bf(M + 1, K))
    with pytest.raises(ValueError, match="on the GPU"):
        g.embedding(M, V, K, t.cpu(), B, A)
    with pytest.raises(TypeError, match="ids: expected"):
        g.embedding(M, V, K, t.float(), B, A)
    with pytest.raises(TypeError, match="E: expected"):
        g.embedding(M, V, K, t, B.half(), A)
    with pytest.raises(ValueError, match="contiguous"):
        g.embedding(M, V, K, t, bf(K, V).t(), A)
    with pytest.raises(TypeError, match="R: expected"):
        g.embedding_bwd(M, V, K, t, A, f(V, K), B, 1.0, ws)
    with pytest.raises(TypeError, match="mean: expected"):
        g.layer_norm(M, K, A, None, None, bf(M, K), bf(2 * M), None)
    with pytest.raises(TypeError, match="beta: expected"):
        g.layer_norm(M, K, A, bf(K), f(K), bf(M, K), None, None)
    with pytest.raises(TypeError, match="Y: expected"):
        g.layer_norm(M, K, A, None, None, f(M, K), None, None)
    with pytest.raises(TypeError, match="dX: expected"):
        g.layer_norm_bwd(M, K, A, None, f(M), f(M), bf(M, K), None, f(M, K), None, None)
    with pytest.raises(g.Gemm355Error) as e:
        g.layer_norm(M, K, A, None, None, A, None, None)
    assert e.value.status == g.ERR_INVALID_ARG
    with pytest.raises(TypeError, match="targets: expected"):
        g.gemm_bf16_nt_cross_entropy(M, V, K, A, B, t.short(), f(M), f(M), ws)
    with pytest.raises(TypeError, match="loss: expected"):
        g.gemm_bf16_nt_cross_entropy(M, V, K, A, B, t, bf(2 * M), f(M), ws)
    with pytest.raises(TypeError, match="A: expected"):
        g.gemm_bf16_nt_cross_entropy(M, V, K, f(M, K), B, t, f(M), f(M), ws)
    with pytest.raises(ValueError, match="workspace_bytes"):
        g.gemm_bf16_nt_cross_entropy(M, V, K, A, B, t, f(M), f(M), ws.data_ptr())
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm_bf16_nt_cross_entropy(M, V, K, A, B, t, f(M), f(M), ws[:64])
    assert e.value.status == g.ERR_UNSUPPORTED
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm_bf16_nt_cross_entropy_bwd(M, V, K, A, B, t, f(M), None, bf(M, K), bf(V, K))
    assert e.value.status == g.ERR_INVALID_ARG
    with pytest.raises(OverflowError):
        g.layer_norm(1 << 40, K, A, None, None, bf(M, K), None, None)
    # what was refused left nothing behind: the next call is right
    g.embedding(M, V, K, t, B, A)
    torch.cuda.synchronize()
    assert not A.any()
