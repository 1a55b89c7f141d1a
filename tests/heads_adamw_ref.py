"""Plain 64-bit restatements of the heads' operators and of AdamW
(include/rot_ops.h), for their tests."""

import math

import numpy as np
import torch

from tests import operators_ref


def angles(turns, positions):
    """float64 radians [.., pairs]: the product modulo 2^64 (int64 wraps) as a part of a turn."""
    part = positions[..., None].to(torch.int64) * turns
    return part.double() * (2 * math.pi / 2.0 ** 64)


def rotated(x, rotary, positions, inverse=False):
    """x [.., tokens, heads, dim] in float64, positions [.., tokens]."""
    x = x.double()
    n = rotary.turns.numel()
    a = angles(rotary.turns, positions)[..., None, :] * (-1 if inverse else 1)
    c, s = rotary.magnitude * torch.cos(a), rotary.magnitude * torch.sin(a)
    y = x.clone()
    i = torch.arange(n, device=x.device)
    u, v = (2 * i, 2 * i + 1) if rotary.interleaved else (i, i + n)
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., v] * c + x[..., u] * s
    return y


def pair_size(x, rotary):
    """|a| + |b| of each element's pair times the magnitude (|x| where it is not rotated), float64."""
    x = x.double().abs()
    if rotary is None:
        return x
    n = rotary.turns.numel()
    i = torch.arange(n, device=x.device)
    u, v = (2 * i, 2 * i + 1) if rotary.interleaved else (i, i + n)
    y = x.clone()
    y[..., u] = y[..., v] = (x[..., u] + x[..., v]) * max(abs(rotary.magnitude), 1e-30)
    return y


def normed(x, w, eps):
    """(x r w, hat, r) in float64."""
    x = x.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * r * w.double(), x * r, r


def norm_grad(g, x, w, eps):
    """(dx, dw) from the gradient g of x r w."""
    _, hat, r = normed(x, w, eps)
    gw = g.double() * w.double()
    dx = r * (gw - hat * (gw * hat).mean(-1, keepdim=True))
    return dx, (g.double() * hat).flatten(0, -2).sum(0)


# ---- AdamW ----


def words(base, count, step, seed):
    """The generator's words of `count` elements of a tensor that begins at element `base` (a multiple of 128)."""
    j = np.arange(base // 4, base // 4 + -(-count // 4), dtype=np.uint64)
    return operators_ref.philox(j, step, seed).reshape(-1)[:count].astype(np.int64)


def scale_exponents(x):
    """Least e >= -127 with all finite elements of each 128 within 448 2^e, one for each element; x: float64 numpy."""
    out = np.zeros(-(-len(x) // 128))
    for i in range(len(out)):
        b = np.abs(x[i * 128:(i + 1) * 128])
        b = b[np.isfinite(b)]
        big = b.max() if len(b) else 0.0
        e = -127
        while big > 448.0 * 2.0 ** e:
            e += 1
        out[i] = e
    return np.repeat(out, 128)[:len(x)]


def grid(x, exponents, bits, least):
    """Steps of the grid of `bits` fraction bits (exponents from `least` up) under 2^exponents, at |x|."""
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(np.isfinite(x), np.abs(x), 0.0) * 2.0 ** -exponents
        k = np.where(y > 0, np.frexp(y)[1], -1000)
    return 2.0 ** (np.maximum(k - 1, least) - bits + exponents)


def step(p, g, m, v, t, lr, beta1, beta2, eps, decay, factor=1.0):
    """(p, m, v) after one step, float64 arrays."""
    g = g * factor
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    u = lr / (1 - beta1 ** t) * m / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p * (1 - lr * decay) - u, m, v
