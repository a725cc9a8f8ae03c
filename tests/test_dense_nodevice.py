"""The layer calls of the C ABI without a GPU: every refusal happens before any
HIP call, so the addresses here are never dereferenced."""
import ctypes

import pytest

import dense_gemm_14_amd as g

A, B, BIAS, R, Z, C, DC, DA, DB, DBIAS, WS = (0x10000 + (i << 24) for i in range(11))
BIG = 1 << 34   # a workspace size that is never too small for the checks below


def linear(M=8, N=8, K=64, a=A, b=B, bias=BIAS, act=0, r=R, z=Z, c=C, ws=None, nb=0):
    return g.load().gemm_bf16_nt_bias_act_res(M, N, K, a, b, bias, act, r, z, c, ws, nb, None)


def gated(M=8, N=8, K=64, a=A, b=B, bias=BIAS, act=0, z=Z, c=C, ws=None, nb=0):
    return g.load().gemm_bf16_nt_gated(M, N, K, a, b, bias, act, z, c, ws, nb, None)


def linear_bwd(M=8, N=8, K=64, a=A, b=B, z=Z, act=0, dc=DC, da=DA, db=DB, dbias=DBIAS, ws=None, nb=0):
    return g.load().gemm_bf16_nt_bias_act_bwd(M, N, K, a, b, z, act, dc, da, db, dbias, ws, nb, None)


def gated_bwd(M=8, N=8, K=64, a=A, b=B, z=Z, act=0, dc=DC, da=DA, db=DB, dbias=DBIAS, ws=None, nb=0):
    return g.load().gemm_bf16_nt_gated_bwd(M, N, K, a, b, z, act, dc, da, db, dbias, ws, nb, None)


def ortho(batch=1, rows=8, cols=8, t=0, G=A, steps=5, a=3.0, b=-4.0, c=2.0, eps=0.0, o=C, ws=WS, nb=1 << 20):
    return g.load().gemm355_newton_schulz(batch, rows, cols, t, G, steps, a, b, c, eps, o, ws, nb, None)


ALL = [linear, gated, linear_bwd, gated_bwd]


@pytest.mark.parametrize("fn", ALL)
def test_sizes_activations_and_workspaces(fn):
    for bad in (dict(M=-1), dict(N=-8), dict(K=-8), dict(act=-1), dict(act=4), dict(ws=None, nb=16)):
        assert fn(**bad) == g.ERR_INVALID_ARG, bad
    # granularity and alignment
    for bad in (dict(N=12), dict(K=12), dict(a=A + 2), dict(b=B + 8), dict(z=Z + 4), dict(ws=WS + 8, nb=64)):
        assert fn(**bad) == g.ERR_UNSUPPORTED, bad
    # an operand of 4 GiB
    assert fn(M=1 << 17, N=8, K=1 << 14, b=1 << 40, z=1 << 41, **{("c" if fn in (linear, gated) else "da"): 1 << 42,
              **({"r": None} if fn is linear else {}), **({"db": 1 << 43, "dbias": 1 << 44, "dc": 1 << 45}
                                                          if fn in (linear_bwd, gated_bwd) else {"bias": None})}) == g.ERR_UNSUPPORTED


@pytest.mark.parametrize("fn", [linear, gated])
def test_forward_pointers_and_overlaps(fn):
    assert fn(c=None) == g.ERR_INVALID_ARG
    assert fn(a=None) == g.ERR_INVALID_ARG
    assert fn(b=None) == g.ERR_INVALID_ARG
    for bad in (dict(c=A + 64), dict(c=B), dict(c=Z + 16), dict(c=BIAS), dict(z=A), dict(z=B + 16), dict(z=BIAS),
                dict(ws=C, nb=1024), dict(ws=Z, nb=1024), dict(ws=A + 16, nb=1024), dict(ws=BIAS, nb=16)):
        assert fn(**bad) == g.ERR_INVALID_ARG, bad
    assert fn(M=0, a=None, b=None, bias=None, z=None, c=None) == g.OK
    assert fn(N=0, a=None, b=None, bias=None, z=None, c=None) == g.OK


def test_residual_may_be_c_itself_and_nothing_else():
    assert linear(r=C + 16) == g.ERR_INVALID_ARG
    assert linear(r=Z) == g.ERR_INVALID_ARG
    assert linear(ws=R, nb=1024) == g.ERR_INVALID_ARG
    assert linear(r=C, ws=C, nb=1024) == g.ERR_INVALID_ARG
    assert linear(r=C, z=C) == g.ERR_INVALID_ARG
    assert linear(r=R + 8) == g.ERR_UNSUPPORTED
    # C == R passes the checks (and then meets the missing device)
    import torch
    if not torch.cuda.is_available():
        assert linear(r=C) == g.ERR_NO_DEVICE


@pytest.mark.parametrize("fn", [linear_bwd, gated_bwd])
def test_backward_pointers_and_overlaps(fn):
    assert fn(dc=None) == g.ERR_INVALID_ARG
    assert fn(act=2, z=None) == g.ERR_INVALID_ARG      # Z is needed
    assert fn(a=None) == g.ERR_INVALID_ARG             # dB needs A
    assert fn(b=None) == g.ERR_INVALID_ARG             # dA needs B
    outs = dict(da=DA, db=DB, dbias=DBIAS)
    for o in outs:
        for other in (A, B, Z, DC, *[v for k, v in outs.items() if k != o]):
            assert fn(**{o: other}) == g.ERR_INVALID_ARG, (o, other)
        assert fn(**{o: outs[o] + 8}) == g.ERR_UNSUPPORTED
    assert fn(ws=DA, nb=1024) == g.ERR_INVALID_ARG
    assert fn(ws=Z, nb=1024) == g.ERR_INVALID_ARG
    # nothing wanted, or nothing to write: fine with no arrays at all
    assert fn(a=None, b=None, z=None, dc=None, da=None, db=None, dbias=None) == g.OK
    assert fn(M=0, N=0, a=None, b=None, z=None, dc=None) == g.OK


def test_newton_schulz_refusals():
    nan, inf = float("nan"), float("inf")
    for bad in (dict(batch=-1), dict(rows=-8), dict(cols=-8), dict(t=2), dict(t=-1), dict(steps=0), dict(steps=65),
                dict(a=nan), dict(b=inf), dict(c=-inf), dict(eps=-1e-9), dict(eps=nan), dict(G=None), dict(o=None),
                dict(ws=None), dict(ws=None, nb=0), dict(o=A), dict(ws=A + 16), dict(ws=C)):
        assert ortho(**bad) == g.ERR_INVALID_ARG, bad
    for bad in (dict(rows=12), dict(cols=20), dict(G=A + 8), dict(o=C + 2), dict(ws=WS + 8),
                dict(rows=1 << 15, cols=1 << 15, G=1 << 40, o=1 << 42, ws=1 << 44), dict(batch=65536, o=1 << 40)):
        assert ortho(**bad) == g.ERR_UNSUPPORTED, bad
    assert ortho(batch=0, G=None, o=None, ws=None) == g.OK
    assert ortho(rows=0, G=None, o=None, ws=None) == g.OK


def test_workspace_size_refusals():
    lib, n = g.load(), ctypes.c_size_t(7)
    for name, args in (("gemm_bf16_nt_bias_act_res", ()), ("gemm_bf16_nt_gated", ()), ("gemm_bf16_nt_gated_bwd", ()),
                       ("gemm_bf16_nt_bias_act_bwd", (0,)), ("gemm355_newton_schulz", ())):
        fn = getattr(lib, name + "_workspace_size")
        for bad in ((-1, 8, 8), (8, -1, 8), (8, 8, -1)):
            assert fn(*bad, *args, ctypes.byref(n)) == g.ERR_INVALID_ARG
        assert fn(8, 8, 8, *args, None) == g.ERR_INVALID_ARG
        assert n.value == 7
        assert fn(0, 0, 0, *args, ctypes.byref(n)) == g.OK and n.value == 0
        n.value = 7
    assert lib.gemm_bf16_nt_bias_act_bwd_workspace_size(8, 8, 8, 4, ctypes.byref(n)) == g.ERR_INVALID_ARG


def test_sizes_beyond_the_limit():
    # the largest ints: refused as too large, with no arithmetic running over
    lib, n, top = g.load(), ctypes.c_size_t(7), (1 << 31) - 8
    for name, args in (("gemm_bf16_nt_bias_act_res", ()), ("gemm_bf16_nt_gated", ()), ("gemm_bf16_nt_gated_bwd", ()),
                       ("gemm_bf16_nt_bias_act_bwd", (0,))):
        fn = getattr(lib, name + "_workspace_size")
        for sizes in ((top, top, top), (8, top, 8), (0, top, 0), (top, 8, 8), (8, 8, top)):
            assert fn(*sizes, *args, ctypes.byref(n)) == g.ERR_UNSUPPORTED, (name, sizes)
    for sizes in ((top, 8, 8), (1, top, top), (65535, 1 << 14, 1 << 14)):
        assert lib.gemm355_newton_schulz_workspace_size(*sizes, ctypes.byref(n)) == g.ERR_UNSUPPORTED, sizes
    assert n.value == 7
    assert linear(M=8, N=top, K=0, a=None, b=None, bias=None, r=None, z=None, c=1 << 45) == g.ERR_UNSUPPORTED
    assert gated_bwd(M=0, N=top, K=0, a=None, b=None, z=None, dc=None, da=None, db=None, dbias=1 << 45) == g.ERR_UNSUPPORTED
    assert ortho(batch=65535, rows=1 << 14, cols=1 << 14, G=1 << 50, o=1 << 52, ws=1 << 54) == g.ERR_UNSUPPORTED


def test_the_older_calls_still_refuse_silu():
    assert g.load().gemm_bf16_nt_bias_act(8, 8, 64, A, B, BIAS, g.ACT_SILU, C, None) == g.ERR_INVALID_ARG
