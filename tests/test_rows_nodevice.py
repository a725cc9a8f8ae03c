"""Embedding, layer norm and cross entropy of the C ABI without a GPU: every refusal happens
before any HIP call, so the addresses here are never dereferenced; and what the
binding refuses before it asks for a device."""
import ctypes

import pytest

import dense_gemm_14_amd as g

IDS, E, Y, R, X, GAMMA, BETA, MEAN, RSTD, DY, DX, DG, DB, WS = (0x10000 + (i << 24) for i in range(14))
TOP = (1 << 31) - 8
INF, NAN = float("inf"), float("nan")


def embed(tokens=8, vocab=16, cols=64, it=1, ids=IDS, et=0, e=E, scale=1.0, yt=0, y=Y):
    return g.load().gemm355_embedding(tokens, vocab, cols, it, ids, et, e, scale, yt, y, None)


def embed_bwd(tokens=8, vocab=16, cols=64, it=1, ids=IDS, yt=0, dy=DY, scale=1.0, et=0, r=R, de=E, ws=WS, nb=1 << 20):
    return g.load().gemm355_embedding_bwd(tokens, vocab, cols, it, ids, yt, dy, scale, et, r, de, ws, nb, None)


def norm(rows=8, cols=64, xt=0, x=X, wt=0, gamma=GAMMA, beta=BETA, eps=1e-5, y=Y, mean=MEAN, rstd=RSTD):
    return g.load().gemm355_layer_norm(rows, cols, xt, x, wt, gamma, beta, eps, y, mean, rstd, None)


def norm_bwd(rows=300, cols=64, xt=0, x=X, wt=0, gamma=GAMMA, mean=MEAN, rstd=RSTD, dy=DY, r=R, dx=DX, dg=DG, db=DB,
             ws=WS, nb=1 << 20):
    return g.load().gemm355_layer_norm_bwd(rows, cols, xt, x, wt, gamma, mean, rstd, dy, r, dx, dg, db, ws, nb, None)


A, B, T, LOSS, LSE, DLOSS = ((64 + i) << 24 for i in range(6))


def entropy(M=80, V=100, K=64, a=A, b=B, tt=1, t=T, loss=LOSS, lse=LSE, ws=WS, nb=1 << 23):
    return g.load().gemm_bf16_nt_cross_entropy(M, V, K, a, b, tt, t, loss, lse, ws, nb, None)


def entropy_bwd(M=80, V=100, K=64, a=A, b=B, tt=1, t=T, lse=LSE, dloss=DLOSS, da=DX, db=DB, ws=WS, nb=1 << 23):
    return g.load().gemm_bf16_nt_cross_entropy_bwd(M, V, K, a, b, tt, t, lse, dloss, da, db, ws, nb, None)


def no_gpu():
    import torch
    return not torch.cuda.is_available()


def test_embedding_refusals():
    for bad in (dict(tokens=-1), dict(vocab=-1), dict(cols=-8), dict(it=2), dict(it=-1), dict(et=2), dict(yt=-1),
                dict(scale=INF), dict(scale=NAN), dict(ids=None), dict(y=None), dict(e=None), dict(y=E + 64),
                dict(y=IDS + 16)):
        assert embed(**bad) == g.ERR_INVALID_ARG, bad
    for bad in (dict(cols=12), dict(e=E + 8), dict(y=Y + 2), dict(ids=IDS + 4), dict(it=0, ids=IDS + 2),
                dict(tokens=TOP, cols=TOP, y=1 << 45), dict(vocab=TOP, cols=TOP)):
        assert embed(**bad) == g.ERR_UNSUPPORTED, bad
    assert embed(tokens=0, ids=None, e=None, y=None) == g.OK
    assert embed(cols=0, ids=None, e=None, y=None) == g.OK
    if no_gpu():   # passes the checks and meets the missing device
        for ok in ({}, dict(vocab=0, e=None), dict(ids=IDS + 8), dict(it=0, ids=IDS + 4), dict(et=1, yt=1)):
            assert embed(**ok) == g.ERR_NO_DEVICE, ok


def test_embedding_gradient_refusals():
    for bad in (dict(tokens=-1), dict(vocab=-1), dict(cols=-8), dict(it=2), dict(et=2), dict(yt=2), dict(scale=NAN),
                dict(ids=None), dict(dy=None), dict(de=None), dict(ws=None), dict(de=DY + 64),
                dict(r=E + 64), dict(de=IDS), dict(ws=E), dict(ws=DY), dict(ws=R), dict(ws=IDS), dict(r=E, ws=E)):
        assert embed_bwd(**bad) == g.ERR_INVALID_ARG, bad
    for bad in (dict(cols=12), dict(dy=DY + 8), dict(de=E + 8), dict(r=R + 8), dict(ws=WS + 8), dict(ids=IDS + 4),
                dict(tokens=TOP, cols=TOP, dy=1 << 45), dict(vocab=TOP, cols=TOP, de=1 << 45, r=None)):
        assert embed_bwd(**bad) == g.ERR_UNSUPPORTED, bad
    assert embed_bwd(vocab=0, ids=None, dy=None, r=None, de=None, ws=None, nb=0) == g.OK
    assert embed_bwd(cols=0, ids=None, dy=None, r=None, de=None, ws=None, nb=0) == g.OK
    if no_gpu():
        for ok in ({}, dict(r=E), dict(r=None), dict(tokens=0, ids=None, dy=None), dict(ws=None, nb=0)):
            assert embed_bwd(**ok) == g.ERR_NO_DEVICE, ok


def test_norm_refusals():
    for bad in (dict(rows=-1), dict(cols=-8), dict(xt=2), dict(wt=-1), dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF),
                dict(x=None), dict(y=None), dict(y=X), dict(mean=X + 16), dict(mean=RSTD), dict(y=GAMMA), dict(rstd=BETA),
                dict(mean=Y + 4)):
        assert norm(**bad) == g.ERR_INVALID_ARG, bad
    for bad in (dict(cols=12), dict(x=X + 8), dict(y=Y + 2), dict(gamma=GAMMA + 8), dict(beta=BETA + 4), dict(mean=MEAN + 2),
                dict(rstd=RSTD + 1), dict(rows=TOP, cols=TOP, x=1 << 45, y=1 << 50, mean=None, rstd=None)):
        assert norm(**bad) == g.ERR_UNSUPPORTED, bad
    assert norm(rows=0, x=None, y=None) == g.OK and norm(cols=0, x=None, y=None) == g.OK
    if no_gpu():
        for ok in ({}, dict(gamma=None, beta=None, mean=None, rstd=None), dict(mean=MEAN + 4, rstd=RSTD + 12)):
            assert norm(**ok) == g.ERR_NO_DEVICE, ok


def test_norm_gradient_refusals():
    for bad in (dict(rows=-1), dict(cols=-8), dict(xt=2), dict(wt=2), dict(x=None), dict(mean=None), dict(rstd=None),
                dict(dy=None), dict(ws=None), dict(dx=X), dict(dx=DY), dict(dx=R + 16), dict(dx=GAMMA), dict(dg=DB),
                dict(dg=X), dict(db=DY), dict(ws=DX), dict(ws=X), dict(ws=MEAN), dict(dg=RSTD), dict(r=DX, dg=DX)):
        assert norm_bwd(**bad) == g.ERR_INVALID_ARG, bad
    for bad in (dict(cols=12), dict(x=X + 8), dict(dy=DY + 8), dict(r=R + 8), dict(dx=DX + 4), dict(dg=DG + 2), dict(ws=WS + 8),
                dict(gamma=GAMMA + 8), dict(mean=MEAN + 2),
                dict(rows=TOP, cols=TOP, x=1 << 45, dy=1 << 50, dx=None, r=None)):
        assert norm_bwd(**bad) == g.ERR_UNSUPPORTED, bad
    # nothing wanted, or nothing to write: fine with no arrays at all
    assert norm_bwd(x=None, mean=None, rstd=None, dy=None, dx=None, dg=None, db=None) == g.OK
    assert norm_bwd(rows=0, x=None, mean=None, rstd=None, dy=None, dg=None, db=None) == g.OK
    assert norm_bwd(cols=0, x=None, mean=None, rstd=None, dy=None) == g.OK
    if no_gpu():
        for ok in ({}, dict(r=DX), dict(r=None), dict(gamma=None), dict(dx=None), dict(dg=None), dict(rows=8, ws=None, nb=0)):
            assert norm_bwd(**ok) == g.ERR_NO_DEVICE, ok


def test_cross_entropy_refusals():
    for bad in (dict(M=-1), dict(V=-1), dict(K=-8), dict(tt=2), dict(tt=-1), dict(a=None), dict(b=None), dict(t=None),
                dict(loss=None), dict(lse=None), dict(ws=None), dict(ws=None, nb=0), dict(loss=LSE), dict(loss=A + 16),
                dict(lse=B), dict(lse=T), dict(ws=A), dict(ws=B), dict(ws=T), dict(ws=LOSS), dict(loss=LSE + 4)):
        assert entropy(**bad) == g.ERR_INVALID_ARG, bad
    for bad in (dict(K=12), dict(a=A + 8), dict(b=B + 2), dict(t=T + 4), dict(tt=0, t=T + 2), dict(loss=LOSS + 2),
                dict(lse=LSE + 1), dict(ws=WS + 8), dict(M=TOP, a=1 << 45, t=1 << 50, loss=1 << 52, lse=1 << 53),
                dict(K=1 << 22, a=1 << 45, b=1 << 50), dict(M=1 << 24, V=TOP, K=8, a=1 << 45, b=1 << 50, t=1 << 52)):
        assert entropy(**bad) == g.ERR_UNSUPPORTED, bad
    assert entropy(M=0, a=None, b=None, t=None, loss=None, lse=None, ws=None, nb=0) == g.OK
    if no_gpu():
        for ok in ({}, dict(V=0, b=None), dict(K=0, a=None, b=None), dict(V=101), dict(t=T + 8), dict(tt=0, t=T + 4),
                   dict(loss=LOSS + 4, lse=LSE + 12)):
            assert entropy(**ok) == g.ERR_NO_DEVICE, ok


def test_cross_entropy_gradient_refusals():
    for bad in (dict(M=-1), dict(V=-1), dict(K=-8), dict(tt=2), dict(a=None), dict(b=None), dict(t=None), dict(lse=None),
                dict(ws=None), dict(ws=None, nb=0), dict(da=A), dict(da=B), dict(db=B), dict(db=A), dict(da=DB), dict(da=T),
                dict(da=LSE), dict(db=DLOSS), dict(ws=A), dict(ws=DX), dict(ws=DB), dict(ws=LSE), dict(ws=DLOSS)):
        assert entropy_bwd(**bad) == g.ERR_INVALID_ARG, bad
    for bad in (dict(K=12), dict(a=A + 8), dict(b=B + 2), dict(da=DX + 8), dict(db=DB + 4), dict(t=T + 4), dict(lse=LSE + 2),
                dict(dloss=DLOSS + 1), dict(ws=WS + 8), dict(M=TOP, a=1 << 45, t=1 << 50, da=None, lse=1 << 52, dloss=None),
                dict(K=1 << 22, a=1 << 45, b=1 << 50, da=None, db=1 << 55)):
        assert entropy_bwd(**bad) == g.ERR_UNSUPPORTED, bad
    none = dict(a=None, b=None, t=None, lse=None, dloss=None, ws=None, nb=0)
    assert entropy_bwd(da=None, db=None, **none) == g.OK
    assert entropy_bwd(K=0, **none) == g.OK
    assert entropy_bwd(M=0, V=0, **none) == g.OK
    assert entropy_bwd(M=0, db=None, **none) == g.OK and entropy_bwd(V=0, da=None, **none) == g.OK
    if no_gpu():
        for ok in ({}, dict(dloss=None), dict(da=None), dict(db=None), dict(V=0, b=None), dict(V=101),
                   dict(M=0, a=None, b=None, t=None, lse=None, dloss=None), dict(lse=LSE + 4, dloss=DLOSS + 4)):
            assert entropy_bwd(**ok) == g.ERR_NO_DEVICE, ok


def test_workspace_size_refusals():
    lib, n = g.load(), ctypes.c_size_t(7)
    for name, count in (("gemm355_embedding_bwd", 3), ("gemm355_layer_norm_bwd", 2), ("gemm_bf16_nt_cross_entropy", 3),
                        ("gemm_bf16_nt_cross_entropy_bwd", 3)):
        fn = getattr(lib, name + "_workspace_size")
        for i in range(count):
            assert fn(*[-1 if j == i else 8 for j in range(count)], ctypes.byref(n)) == g.ERR_INVALID_ARG
        assert fn(*[8] * count, None) == g.ERR_INVALID_ARG
        assert fn(*[TOP] * count, ctypes.byref(n)) == g.ERR_UNSUPPORTED
        assert n.value == 7
        assert fn(*[0] * count, ctypes.byref(n)) == g.OK and n.value == 0
        n.value = 7


def test_binding_refuses_before_it_asks_for_a_device():
    import torch
    f32, bf16, i64 = (torch.zeros(64, dtype=t) for t in (torch.float32, torch.bfloat16, torch.int64))
    for bad in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(TypeError, match="X: expected"):
            g._type_of(None, "X", torch.zeros(8, dtype=bad))
    with pytest.raises(ValueError, match="raw address"):
        g._type_of(None, "X", 64)
    with pytest.raises(ValueError, match="BF16 or FP32"):
        g._type_of(2, "X", 64)
    with pytest.raises(OverflowError):
        g._type_of(1 << 32, "X", 64)
    assert g._type_of(None, "X", None, f32) == g.FP32 and g._type_of(None, "X", bf16, f32) == g.BF16
    assert g._type_of(None, "X", None) == g.BF16 and g._type_of(g.FP32, "X", 64) == g.FP32
    with pytest.raises(TypeError, match="Y: expected"):
        g._values(f32, g.BF16, 8, "Y", 0)
    with pytest.raises(TypeError, match="Y: expected"):
        g._values(bf16, g.FP32, 8, "Y", 0)
    with pytest.raises(TypeError, match="mean: expected"):
        g._floats(bf16, 8, "mean", 0)
    for bad in (torch.int16, torch.float32, torch.uint8, torch.bool):
        with pytest.raises(TypeError, match="ids: expected"):
            g._ids(torch.zeros(8, dtype=bad), None, 8, "ids", 0)
    with pytest.raises(ValueError, match="raw address"):
        g._ids(64, None, 8, "ids", 0)
    with pytest.raises(ValueError, match="on the GPU"):
        g._ids(i64, None, 8, "ids", 0)
    assert g._ids(64, g.INT64, 8, "ids", 0) == (64, g.INT64) and g._ids(None, None, 0, "ids", 0) == (None, 0)


@pytest.mark.parametrize("far", [1 << 31, 1 << 32, -(1 << 32) + 8])
def test_sizes_beyond_32_bits_are_refused(far):
    for i in range(3):
        with pytest.raises(OverflowError):
            g.embedding(*[far if j == i else 8 for j in range(3)], 64, 64, 64, id_type=0, e_type=0, y_type=0)
        with pytest.raises(OverflowError):
            g.embedding_bwd(*[far if j == i else 8 for j in range(3)], 64, 64, None, 64, id_type=0, e_type=0, y_type=0)
        with pytest.raises(OverflowError):
            g.embedding_bwd_workspace_size(*[far if j == i else 8 for j in range(3)])
        with pytest.raises(OverflowError):
            g.gemm_bf16_nt_cross_entropy(*[far if j == i else 8 for j in range(3)], 64, 64, 64, 64, 64, target_type=0)
        with pytest.raises(OverflowError):
            g.gemm_bf16_nt_cross_entropy_bwd(*[far if j == i else 8 for j in range(3)], 64, 64, 64, 64, 64, 64, 64,
                                             target_type=0)
        with pytest.raises(OverflowError):
            g.cross_entropy_workspace_size(*[far if j == i else 8 for j in range(3)])
        with pytest.raises(OverflowError):
            g.cross_entropy_bwd_workspace_size(*[far if j == i else 8 for j in range(3)])
    for i in range(2):
        with pytest.raises(OverflowError):
            g.layer_norm(*[far if j == i else 8 for j in range(2)], 64, None, None, 64, None, None, x_type=0)
        with pytest.raises(OverflowError):
            g.layer_norm_bwd(*[far if j == i else 8 for j in range(2)], 64, None, 64, 64, 64, None, 64, None, None, x_type=0)
        with pytest.raises(OverflowError):
            g.layer_norm_bwd_workspace_size(*[far if j == i else 8 for j in range(2)])
