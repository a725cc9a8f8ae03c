"""Every choice of gradients of a layer's backward call: dA, dB and dbias, alone
and together, linear and gated, with whole numbers whose sums are exact in FP32,
so each output has one right value. The sizes make a lone product take 64 x 64
tiles with eight, four, two waves and one, narrow ones, 128 x 128 and 256 x 256."""
import itertools

import pytest
import torch

import dense_gemm_14_amd as g
from tests.dense_util import GUARD, Out, workspace
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

SIZES = [(1, 4096, 4096), (8, 4096, 4096), (64, 4096, 4096), (64, 2048, 2048), (1310, 168, 6288), (1310, 6288, 168),
         (4096, 128, 4096), (301, 1384, 512), (777, 1000, 520), (2050, 2056, 1032), (37, 8, 72)]
WANTED = [w for n in (1, 2, 3) for w in itertools.combinations(("dA", "dB", "dbias"), n)]


def whole(gen, *shape, top=2):
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").to(torch.bfloat16)


def right(out, want, what):
    """The device array holds `want` and the bands around it are untouched."""
    assert torch.equal(out.t, want), "%s: %d of %d differ" % (what, int((out.t != want).sum()), want.numel())
    assert (out.buf[:GUARD] == 0x7FC1).all() and (out.buf[GUARD + out.n:] == 0x7FC1).all(), "write outside %s" % what


@pytest.mark.parametrize("choice", [g.LAYER_AUTO, g.LAYER_SMALL], ids=["auto", "small"])
@pytest.mark.parametrize("gated,act", [(False, g.ACT_NONE), (False, g.ACT_RELU), (True, g.ACT_RELU)],
                         ids=["linear", "relu", "gated"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_every_choice_of_gradients_is_exact(choice, gated, act, M, N, K):
    need_gpu()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M + N)
    rows = 2 * N if gated else N
    A, B, Z, dC = whole(gen, M, K), whole(gen, rows, K), whole(gen, M, rows), whole(gen, M, N, top=1)
    z, dz = Z.float(), dC.float()
    if gated:
        dz = torch.cat([dz * z[:, N:] * (z[:, :N] > 0), dz * z[:, :N].clamp(min=0)], 1)
    elif act == g.ACT_RELU:
        dz = dz * (z > 0)
    want = {"dA": (dz @ B.float()).bfloat16(), "dB": (dz.t().contiguous() @ A.float()).bfloat16(),
            "dbias": dz.sum(0).bfloat16()}
    call = g.gemm_bf16_nt_gated_bwd if gated else g.gemm_bf16_nt_bias_act_bwd
    g.force_layer_kernel(choice)
    try:
        ws, nb, check = workspace(g.gated_bwd_workspace_size(M, N, K) if gated else
                                  g.bias_act_bwd_workspace_size(M, N, K, act))
        for wanted in WANTED:
            print("gradients", choice, gated, act, M, N, K, wanted, flush=True)
            outs = {"dA": Out(M, K), "dB": Out(rows, K), "dbias": Out(rows)}
            call(M, N, K, A if "dB" in wanted else None, B if "dA" in wanted else None, Z if gated or act else None, act,
                 dC, *[outs[k].t if k in wanted else None for k in outs], ws, nb)
            torch.cuda.synchronize()
            for k in wanted:
                right(outs[k], want[k], k)
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)
    check()
