"""The fused and grouped products' definitions in 64 bits, with error bounds.

Bounds, for a product of K terms with magnitude mag = |alpha| sum |a b| + |bias|:
  e_u = (K + 8) 2^-23 mag     the fp32 sum in any order, each addition rounded or cut
                              (relative error up to 2^-23), alpha and the bias
  act   Lipschitz constant 1.13 (gelu's largest slope), and its evaluation, 2^-22 |u|
  slope evaluated within 2^-20
  out   half a step of the type, and half of its smallest subnormal
"""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def phi(x):
    return 0.5 * torch.erfc(-x / math.sqrt(2.0))


def act(u, name):
    return u * phi(u) if name == "gelu" else torch.relu(u) if name == "relu" else u


def slope(u, name):
    if name == "gelu":
        return phi(u) + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    return (u > 0).double() if name == "relu" else torch.ones_like(u)


def product(a, b, alpha=1.0, bias=None):
    """alpha a @ b + bias of 64-bit values and e_u."""
    p, mag = alpha * (a @ b), abs(alpha) * (a.abs() @ b.abs())
    if bias is not None:
        p, mag = p + bias, mag + bias.abs()
    return p, (a.shape[1] + 8) * 2.0 ** -23 * mag


def rounding(y, dtype):
    return torch.finfo(DT[dtype]).eps / 2 * y.abs() + TINY[dtype]


def forward(a, b, dtype, alpha=1.0, bias=None, name="none", residual=None, beta=1.0):
    """(U, its bound, Y, its bound) of 64-bit a [M, K], b [K, N]."""
    u, eu = product(a, b, alpha, bias)
    y = act(u, name)
    ey = 1.13 * eu + 2.0 ** -22 * u.abs()
    if residual is not None:
        ey = ey + 2.0 ** -22 * (y.abs() + abs(beta) * residual.abs())
        y = y + beta * residual
    return u, eu + rounding(u.abs() + eu, dtype), y, ey + rounding(y.abs() + ey, dtype)


def backward(a, b, dtype, u, alpha=1.0, name="gelu"):
    """(dX, its bound, column sums, their bound)."""
    p, ep = product(a, b, alpha)
    d = p * slope(u, name)
    e = 1.13 * ep + 2.0 ** -20 * p.abs()
    if name == "relu":
        e = torch.where(u > 0, e, 0.0)
    db = d.sum(dim=0)
    edb = e.sum(dim=0) + (a.shape[0] + 8) * 2.0 ** -23 * d.abs().sum(dim=0)
    return d, e + rounding(d.abs() + e, dtype), db, edb


def check(got, want, bound, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)  # (a NaN is bad)
    assert not bad.any(), (what, int(bad.sum()), float((off / bound).nan_to_num(1e30).max()),
                           bad.nonzero()[:4].tolist())
