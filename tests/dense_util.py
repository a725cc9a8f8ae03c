"""Inputs, 64-bit references and error bounds of the layer calls' GPU tests.

Bounds, per element, with u = 2^-8 the half-step of BF16 and v = 2^-24 that of
FP32 (both relative to the value):
  a sum of K products in FP32     K v S,  S = sum |a b| (any order)
  an activation                   its slope times its argument's error, plus
                                  2^-18 (1 + |z|) for the exponential and the
                                  reciprocal
  a value stored in BF16          u |value|
"""
import math

import numpy as np
import torch

U, V = 2.0 ** -8, 2.0 ** -24
GUARD = 4096
SLOPE = {0: 1.0, 1: 1.0, 2: 1.13, 3: 1.1}     # the activations' largest slopes
BEND = {0: 0.0, 1: 0.0, 2: 1.2, 3: 0.51}      # and the largest change of slope per unit of z


class Out:
    """A BF16 device array between two bands of NaN patterns."""

    def __init__(self, *shape, fill=None):
        n = math.prod(shape)
        self.n, self.shape = n, shape
        self.buf = torch.full((n + 2 * GUARD,), 0x7FC1, dtype=torch.int16, device="cuda")
        self.t = self.buf[GUARD:GUARD + n].view(torch.bfloat16).view(*shape)
        if fill is not None:
            self.t.copy_(fill)

    def get(self):
        host = self.buf.cpu()
        assert (host[:GUARD] == 0x7FC1).all() and (host[GUARD + self.n:] == 0x7FC1).all(), "write outside the array"
        return host[GUARD:GUARD + self.n].view(torch.bfloat16).view(*self.shape).double()


def workspace(nbytes):
    """(tensor, check): a workspace filled with NaN patterns and a band after it."""
    buf = torch.full((nbytes // 2 + GUARD,), 0x7FC1, dtype=torch.int16, device="cuda")

    def check():
        assert (buf[(nbytes + 1) // 2:].cpu() == 0x7FC1).all(), "write past the workspace"
    return (buf if nbytes else None), nbytes, check


def randn(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, dtype=torch.float64) * std).to(torch.bfloat16)


def ints(gen, *shape, top=2):
    """Small whole numbers: every sum of their products below 2^24 is exact."""
    return torch.randint(-top, top + 1, shape, generator=gen).to(torch.bfloat16)


def act(name, z):
    if name == 1:
        return torch.clamp(z, min=0)
    if name == 2:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == 3:
        return z * torch.sigmoid(z)
    return z


def slope(name, z):
    z = z.clone().requires_grad_()
    if name == 1:
        return (z > 0).double()
    g, = torch.autograd.grad(act(name, z).sum(), z)
    return g


def act_err(name, z):
    return 2.0 ** -18 * (1 + z.abs()) if name >= 2 else torch.zeros_like(z)


def forward(A, B, bias, name, R, gated):
    """(C, bound of C, Z, bound of Z) of a layer."""
    a, b = A.double(), B.double()
    z = a @ b.t()
    s = a.abs() @ b.abs().t()
    if bias is not None:
        z, s = z + bias.double(), s + bias.double().abs()
    ez = (a.shape[1] + 1) * V * s
    if gated:
        n = z.shape[1] // 2
        zg, zu, eg, eu = z[:, :n], z[:, n:], ez[:, :n], ez[:, n:]
        f = act(name, zg)
        y = f * zu
        ef = SLOPE[name] * eg + act_err(name, zg)
        e = ef * (zu.abs() + eu) + f.abs() * eu + V * y.abs()
    else:
        y = act(name, z)
        e = SLOPE[name] * ez + act_err(name, z)
        if R is not None:
            y = y + R.double()
            e = e + V * (y.abs() + R.double().abs())
    return y, e + U * (y.abs() + e), z, ez + U * (z.abs() + ez)


def backward(A, B, Z, name, dC, gated):
    """{output: (value, bound)} of a layer's gradients."""
    a, b, dc = A.double(), B.double(), dC.double()
    if gated:
        z = Z.double()
        n = z.shape[1] // 2
        zg, zu = z[:, :n], z[:, n:]
        sl, f = slope(name, zg), act(name, zg)
        err = 4 * act_err(name, zg)
        dz = torch.cat([dc * zu * sl, dc * f], 1)
        ed = torch.cat([(dc * zu).abs() * err, dc.abs() * err], 1)
    elif name:
        z = Z.double()
        dz = dc * slope(name, z)
        ed = dc.abs() * 4 * act_err(name, z)
    else:
        dz, ed = dc, torch.zeros_like(dc)
    ed = ed + (3 * V * dz.abs() if gated or name else 0)
    er = ed + (U * (dz.abs() + ed) if gated or name else 0)     # rounded for the products

    def prod(x, ex, y):
        v = x @ y
        e = ex @ y.abs() + (x.shape[1] + 1) * V * ((x.abs() + ex) @ y.abs())
        return v, e + U * (v.abs() + e)
    db = dz.sum(0)
    eb = ed.sum(0) + dz.shape[0] * V * dz.abs().sum(0)
    return {"dA": prod(dz, er, b), "dB": prod(dz.t().contiguous(), er.t().contiguous(), a),
            "dbias": (db, eb + U * (db.abs() + eb))}


def close(got, want, bound, what):
    bad = ~((got - want).abs() <= bound)      # NaN fails
    assert not bad.any(), "%s: %d of %d off, first at %s: got %r, want %r, bound %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item(),
        bound[bad][0].item())
