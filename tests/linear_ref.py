"""The feed-forward operators from their definitions, in 64 bits, and bounds on
how far a result computed in 32 bits and rounded once may be from them.

A sum of n products whose terms' magnitudes add up to S is off by at most
n * 2^-23 * S when every addition may lose a whole unit in the last place of a
32-bit value (the products themselves are exact for 16-bit inputs, and lose
half a unit for 32-bit ones).  A rounding to type t is off by eps(t) / 2 of the
value, and below the smallest normal value by half its smallest step.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -23
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu_erf": 3, "gelu_tanh": 4}
# largest slope of each activation, and largest change of the slope (the second
# derivative's maximum: 1/2 for SiLU, 2 phi(0) = 0.798 and about 0.81 for GELU)
SLOPE = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu_erf": 1.13, "gelu_tanh": 1.13}


def act(name, z):
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu_erf":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid((8 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return z


def slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    with torch.enable_grad():
        x = z.detach().clone().requires_grad_()
        return torch.autograd.grad(act(name, x).sum(), x)[0]


def rounding(t, dtype):
    """Largest error of rounding t's values to dtype."""
    f = torch.finfo(dtype)
    return (f.eps / 2) * t.abs() + f.smallest_normal * f.eps / 2


def linear(X, W, b, R, name):
    """(Y, Z, bound of Z before its rounding)."""
    x, w = X.double(), W.double()
    z = x @ w.t()
    bound = X.shape[1] * U32 * (x.abs() @ w.abs().t())
    if b is not None:
        z = z + b.double()
        bound = bound + U32 * (z.abs() + bound)
    y = act(name, z)
    return (y if R is None else y + R.double()), z, bound


def linear_bound(y, z, zb, R, name, dtype):
    """Bound of Y: the sum's, carried through the activation, 8 units of its own
    evaluation (exponential, division, products), the residual's addition, and
    the rounding."""
    f = SLOPE[name] * zb + 8 * U32 * (act(name, z).abs() + zb)
    if name == "none":
        f = zb
    if R is not None:
        f = f + U32 * (y.abs() + f)
    return f + rounding(y.abs() + f, dtype)


def backward(dY, X, W, Z, name):
    g = dY.double()
    if name != "none":
        g = g * slope(name, Z.double())
    return g @ W.double(), g.t() @ X.double(), g.sum(0), g


def grad_bound(g, dY, name, dtype, parts):
    """Bound of G as the products read it: 16 units of the slope's evaluation
    (relative to dY: a slope is at most 1.13 and may be a difference), and the
    rounding to dtype (twice over where it is held in two parts)."""
    e = torch.zeros_like(g)
    if name in ("none", "relu"):
        return e
    e = 16 * U32 * 1.13 * dY.double().abs()
    if dtype != torch.float32:
        r = rounding(g.abs() + e, dtype)
        e = e + (rounding(r, dtype) if parts else r)
    return e


def moe(X, Wr, W1, W2, k, name, gated, renorm):
    """(Y, ids, weights, bound of Y before its rounding)."""
    x = X.double()
    T, D = x.shape
    F = W2.shape[2]
    logits = x @ Wr.double().t()
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    p = torch.softmax(logits, 1).gather(1, ids)
    if renorm:
        p = p / p.sum(1, keepdim=True)
    Y, B = torch.zeros_like(x), torch.zeros_like(x)
    small = torch.finfo(X.dtype)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            w1, w2 = W1[e].double(), W2[e].double()
            a = w1 @ x[t]
            ab = D * U32 * (w1.abs() @ x[t].abs())
            f = act(name, a[:F])
            fb = SLOPE[name] * ab[:F] + 8 * U32 * (f.abs() + ab[:F])
            if gated:
                h = f * a[F:]
                hb = f.abs() * ab[F:] + (a[F:].abs() + ab[F:]) * fb + U32 * h.abs()
            else:
                h, hb = f, fb
            if X.dtype != torch.float32:   # two parts of the type
                hb = hb + rounding(rounding(h.abs() + hb, X.dtype), X.dtype)
            v = w2 @ h
            vb = w2.abs() @ hb + 2 * F * U32 * (w2.abs() @ (h.abs() + hb))
            Y[t] += p[t, j] * v
            B[t] += p[t, j] * (vb + 3 * U32 * (v.abs() + vb))
    B = B + k * U32 * (Y.abs() + B)
    return Y, ids, p, B
