"""Plain restatements, in 64 bits, of the operators of layers in 16 bits, and
the bounds that their results are held to. They hold none of the library's
code."""

from __future__ import annotations

import math

import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")   # by their SGEMM_ACT_* numbers
JOINS = ("none", "add", "mul")


def half_step(dtype):
    """A rounding to dtype, relative."""
    return torch.finfo(dtype).eps / 2


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def product(a, b):
    """(a . b, sum |a b|) of float64 matrices."""
    return a @ b, a.abs() @ b.abs()


def sum_error(S, n):
    """A sum of n products that are exact in FP32 (two bfloat16 values), S = sum of their magnitudes: n additions, each
    allowed a truncation to 24 bits (2^-23) of at most S; the bias is one more, and the sums of parts of K n / 512 more."""
    return (n + n // 512 + 2) * 2.0 ** -23 * S


# The activations' slopes are at most 1.13 in magnitude (gelu; silu 1.1). Their own evaluation in FP32: silu and gelu_tanh
# are z times a sigmoid, whose exponential is off by 4 * 2^-24 of itself and by its argument's rounding (4 * 2^-24 of the
# argument; |x s(x) (1 - s(x))| <= 0.23), its sum, reciprocal and product by 2 * 2^-24 each; gelu's integral is within
# 1.5e-7 / 2 < 2 * 2^-24 by its formula, its six operations on values of at most 1 within 8 * 2^-24 and its exponential as
# above (|x^2 exp(-x^2 / 2)| <= 0.74). Together below 16 * 2^-24 |z|; twice that is allowed.
ACT_SLOPE = 1.13
ACT_ERROR = 32.0 * 2.0 ** -24


def epilogue(z, e, name, join, D, dtype):
    """(C, its bound, pre's bound) from z in 64 bits with an error of at most e."""
    half = half_step(dtype)
    y = act(z, name)
    e_y = e if name == "none" else ACT_SLOPE * e + ACT_ERROR * z.abs()
    if join == "add":
        c, e_c = y + D, e_y + 2.0 ** -24 * (y.abs() + D.abs() + e_y)
    elif join == "mul":
        c, e_c = y * D, e_y * D.abs() + 2.0 ** -24 * (y.abs() + e_y) * D.abs()
    else:
        c, e_c = y, e_y
    tiny = 2.0 ** -126     # what is below the normal numbers
    return c, e_c + half * (c.abs() + e_c) + tiny, e + half * (z.abs() + e) + tiny


def close(got, want, bound, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= bound) & ~(torch.isnan(got) & torch.isnan(want)) & ~(got == want)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item(),
                                 bound[bad][0].item() if bound.shape == bad.shape else None)


def rms_norm(s, w, eps):
    i = 1.0 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s * i * (w if w is not None else 1.0)


def rms_norm_backward(g, s, w, eps, gs):
    i = 1.0 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    h, gw = s * i, g * (w if w is not None else 1.0)
    d = i * (gw - h * (gw * h).mean(1, keepdim=True))
    return d if gs is None else d + gs, (g * h).sum(0)
