"""Inputs, 64-bit references and error bounds of the tests of embedding and layer
norm.

Bounds, per element, with u the half-step of the stored type (BF16 2^-8, FP32
2^-24, relative to the value) and v = 2^-24 that of FP32:
  a sum in FP32        d v S, S the sum of its terms' magnitudes, d the longest
                       chain of additions that a term passes through
  an FP32 operation    v |result|
  a stored value       u |value|
Row sums: a lane adds up to 64 values (eight at a time for each 8192 columns of a
wide row), then six steps join a wave and at most sixteen more the waves.
"""
import math

import torch

V = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BAND = 512


class Array:
    """A device array between two bands of NaN, with `offset` elements before it
    so that its alignment can be chosen."""

    def __init__(self, *shape, dtype=torch.bfloat16, fill=None):
        n = math.prod(shape)
        self.n = n
        self.buf = torch.full((n + 2 * BAND,), float("nan"), dtype=dtype, device="cuda")
        self.t = self.buf[BAND:BAND + n].view(*shape)
        if fill is not None:
            self.t.copy_(fill)

    def get(self):
        host = self.buf.cpu()
        assert host[:BAND].isnan().all() and host[BAND + self.n:].isnan().all(), "write outside the array"
        return host[BAND:BAND + self.n].view(self.t.shape).double()


def randn(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, dtype=torch.float64) * std).to(dtype)


def chain(cols):
    return 96 + cols // 8192


def stored(value, err, dtype):
    return err + HALF_STEP[dtype] * (value.abs() + err)


def embed(ids, E, scale, vocab, dtype):
    s = torch.tensor(scale, dtype=torch.float32).double()
    kept = (ids >= 0) & (ids < vocab)
    y = torch.zeros(len(ids), E.shape[1], dtype=torch.float64)
    y[kept] = s * E[ids[kept].long()].double()
    return y, stored(y, V * y.abs(), dtype)


def embed_bwd(ids, dY, R, scale, vocab, dtype):
    s = torch.tensor(scale, dtype=torch.float32).double()
    kept = (ids >= 0) & (ids < vocab)
    at, rows = ids[kept].long(), dY[kept].double()
    total = torch.zeros(vocab, dY.shape[1], dtype=torch.float64).index_add_(0, at, rows)
    size = torch.zeros_like(total).index_add_(0, at, rows.abs())
    count = torch.bincount(at, minlength=vocab).double()[:, None]
    out = s * total
    err = s.abs() * size * V * (count + 2)
    if R is not None:
        out = out + R.double()
        err = err + V * (out.abs() + err)
    return out, stored(out, err, dtype)


def norm(X, gamma, beta, eps):
    """{output: (value, bound)} of layer norm."""
    x, d = X.double(), chain(X.shape[1])
    eps = torch.tensor(eps, dtype=torch.float32).double()
    mean = x.mean(1, keepdim=True)
    e_mean = d * V * x.abs().mean(1, keepdim=True) + V * mean.abs()
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    # differences from a mean that is off by e_mean, and the join of the waves'
    e_var = var * (d + 10) * V + 4 * var.sqrt() * e_mean + 4 * e_mean ** 2
    rstd = 1 / torch.sqrt(var + eps)
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 4 * V)
    u = (x - mean) * rstd
    e_u = (V * (x - mean).abs() + e_mean) * rstd + u.abs() * (e_rstd / rstd + V)
    w = gamma.double() if gamma is not None else torch.ones(X.shape[1], dtype=torch.float64)
    b = beta.double() if beta is not None else torch.zeros(X.shape[1], dtype=torch.float64)
    y = u * w + b
    e_y = e_u * w.abs() + V * ((u * w).abs() + y.abs())
    return {"Y": (y, stored(y, e_y, torch.bfloat16)), "mean": (mean[:, 0], e_mean[:, 0]),
            "rstd": (rstd[:, 0], e_rstd[:, 0])}


def norm_bwd(X, gamma, mean, rstd, dY, R, wtype):
    """{output: (value, bound)} of layer norm's gradients, mean and rstd as given."""
    x, dy, m, r = X.double(), dY.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, n = x.shape
    d = chain(n)
    w = gamma.double() if gamma is not None else torch.ones(n, dtype=torch.float64)
    u, g = (x - m) * r, dy * w
    e_u = 3 * V * u.abs()
    sg, su = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
    e_sg = (d + 3) * V * g.abs().mean(1, keepdim=True)
    e_su = (d + 8) * V * (g * u).abs().mean(1, keepdim=True)
    dx = r * (g - sg - u * su)
    parts = g.abs() + sg.abs() + (u * su).abs()
    e_dx = r * (e_sg + u.abs() * e_su + e_u * su.abs() + 4 * V * parts) + V * dx.abs()
    if R is not None:
        dx = dx + R.double()
        e_dx = e_dx + V * dx.abs()
    t = dy * u
    dg, db = t.sum(0), dy.sum(0)
    e_dg, e_db = (rows + 6) * V * t.abs().sum(0), rows * V * dy.abs().sum(0)
    return {"dX": (dx, stored(dx, e_dx, X.dtype)), "dgamma": (dg, stored(dg, e_dg, wtype)),
            "dbeta": (db, stored(db, e_db, wtype))}
