"""The layer calls refuse tensors that hold another type than they compute with,
argument by argument, and take BF16 values held as their bits."""
import pytest
import torch

import dense_gemm_14_amd as g
from tests.dense_util import randn
from tests.gpu_util import need_gpu
from tests.test_gpu_dense import gen_of

pytestmark = pytest.mark.gpu
M, N, K = 24, 40, 72


def arrays(gated):
    gen = gen_of(111, gated)
    rows = 2 * N if gated else N
    t = dict(A=(M, K), B=(rows, K), bias=(rows,), R=(M, N), Z=(M, rows), C=(M, N), dC=(M, N), dA=(M, K), dB=(rows, K),
             dbias=(rows,))
    return {k: randn(gen, *s).cuda() for k, s in t.items()}


def calls(gated, t):
    """(argument names, call) of the forward and the backward call."""
    act, ws = g.ACT_SILU, torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    if gated:
        return [(("A", "B", "bias", "Z", "C"), lambda t: g.gemm_bf16_nt_gated(
            M, N, K, t["A"], t["B"], t["bias"], act, t["Z"], t["C"], ws)),
            (("A", "B", "Z", "dC", "dA", "dB", "dbias"), lambda t: g.gemm_bf16_nt_gated_bwd(
                M, N, K, t["A"], t["B"], t["Z"], act, t["dC"], t["dA"], t["dB"], t["dbias"], ws))]
    return [(("A", "B", "bias", "R", "Z", "C"), lambda t: g.gemm_bf16_nt_bias_act_res(
        M, N, K, t["A"], t["B"], t["bias"], act, t["R"], t["Z"], t["C"], ws)),
        (("A", "B", "Z", "dC", "dA", "dB", "dbias"), lambda t: g.gemm_bf16_nt_bias_act_bwd(
            M, N, K, t["A"], t["B"], t["Z"], act, t["dC"], t["dA"], t["dB"], t["dbias"], ws))]


@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_layers_refuse_other_types(gated):
    need_gpu()
    t = arrays(gated)
    before = {k: v.clone() for k, v in t.items()}
    for names, call in calls(gated, t):
        for name in names:
            for other in (torch.float32, torch.float16):
                with pytest.raises(TypeError, match="%s: expected" % name):
                    call({**t, name: t[name].to(other)})
    torch.cuda.synchronize()
    assert all(torch.equal(t[k], before[k]) for k in t), "a refused call wrote something"
    # the same bits under an integer type: the same results
    for names, call in calls(gated, t):
        call(t)
        bits = {k: v.clone().view(torch.int16) for k, v in t.items()}
        call(bits)
        torch.cuda.synchronize()
        assert all(torch.equal(bits[k], t[k].view(torch.int16)) for k in names)


def test_newton_schulz_refuses_other_types():
    need_gpu()
    G = randn(gen_of(113), 2, 64, 72).cuda()
    O, ws = torch.empty_like(G), torch.empty(g.newton_schulz_workspace_size(2, 64, 72), dtype=torch.uint8, device="cuda")
    for o in (O.float(), O.half()):
        with pytest.raises(TypeError, match="O: expected"):
            g.newton_schulz(2, 64, 72, G, o, workspace=ws)
    with pytest.raises(TypeError, match="G: expected"):
        g.newton_schulz(2, 64, 72, G.float(), O, workspace=ws, g_type=g.BF16)
    with pytest.raises(TypeError, match="G: expected"):
        g.newton_schulz(2, 64, 72, G, O, workspace=ws, g_type=g.FP32)
    g.newton_schulz(2, 64, 72, G, O, workspace=ws)
    bits = torch.empty_like(O, dtype=torch.int16)
    g.newton_schulz(2, 64, 72, G.view(torch.int16), bits, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(bits, O.view(torch.int16))
