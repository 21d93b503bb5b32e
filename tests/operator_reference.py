"""Plain 64-bit implementations of the feed-forward operators and the error
bounds their tests use.  Nothing here uses the product's code.

U is fp32's unit roundoff 2^-24; u_out(dtype) is the output type's, half an ulp
at a power of two relative to it (2^-p for p significant bits), and tiny(dtype)
half its smallest subnormal.
"""

import math

import numpy as np
import torch

U = 2.0 ** -24
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def u_out(dtype):
    return {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U}[dtype]


def tiny(dtype):
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]


def layer_norm(x, w, b, eps):
    x = x.double()
    mean = x.sum(-1, keepdim=True) / x.shape[-1]
    var = (x - mean).square().sum(-1, keepdim=True) / x.shape[-1]
    r = 1 / torch.sqrt(var + eps)
    y = (x - mean) * r
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean[..., 0], r[..., 0]


def layer_norm_backward(dy, x, mean, rstd, w):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    q = dy * w.double() if w is not None else dy
    dx = rstd * (q - q.mean(-1, keepdim=True) - xh * (q * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def chain(width):
    """Longest chain of fp32 additions behind a row sum: up to 32 values a thread (more in very wide rows), 5 steps
    within a warp, up to 32 warps."""
    return (max(32, width / 1024) + 5 + 32 + 2) * U


def layer_norm_bound(x, w, b, eps):
    """|y - exact| of an fp32 evaluation rounded once.  The mean is off by chain * mean|x| and each difference by
    another 4 U |x|; the variance by chain relatively, so rstd by half of that, and a few roundings follow."""
    y, mean, r = layer_norm(x, w, b, eps)
    xd = x.double()
    c = chain(x.shape[-1])
    wd = w.double().abs() if w is not None else torch.ones((), dtype=torch.float64)
    xh = (xd - mean[..., None]) * r[..., None]
    off = wd * (r[..., None] * (c * xd.abs().mean(-1, keepdim=True) + 4 * U * xd.abs()) + (c + 6 * U) * xh.abs())
    return off + 4 * U * (y.abs() + (b.double().abs() if b is not None else 0)) + u_out(x.dtype) * y.abs() * 1.01 + tiny(x.dtype)


def layer_norm_backward_bounds(dy, x, mean, rstd, w):
    """Bounds of dx, dweight and dbias: each product carries a few U, each row mean chain times the mean of absolute
    values, each column sum (rows + 64) U times the sum of absolute values."""
    dx, dw, db = layer_norm_backward(dy, x, mean, rstd, w)
    dyd, xd, m, r = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = ((xd - m) * r).abs()
    q = (dyd * w.double() if w is not None else dyd).abs()
    c = chain(x.shape[-1]) + 8 * U
    dxb = r * (4 * U * q + c * q.mean(-1, keepdim=True) + 2 * c * xh * (q * xh).mean(-1, keepdim=True))
    wt = w.dtype if w is not None else x.dtype
    rows = (x.shape[0] + 64) * U
    return (dxb + u_out(x.dtype) * dx.abs() * 1.01 + tiny(x.dtype),
            (rows + 4 * U) * (dyd.abs() * xh).sum(0) + u_out(wt) * dw.abs() * 1.01 + tiny(wt),
            rows * dyd.abs().sum(0) + u_out(wt) * db.abs() * 1.01 + tiny(wt))


def philox4x32(counter, key, rounds=10):
    """One Philox4x32 block on Python integers (Salmon, Moraes, Dror and Shaw, 2011)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_kept(first, n, p, seed, offset):
    """Whether elements first .. first + n - 1 are kept, as a bool array."""
    low, t = 0xFFFFFFFF, round(p * 2 ** 32)
    words, blocks = [], range(first // 4, (first + n + 3) // 4)
    for b in blocks:
        words += philox4x32((b & low, b >> 32, offset & low, offset >> 32 & low), (seed & low, seed >> 32 & low))
    skip = first - 4 * (first // 4)
    return np.array([w >= t for w in words[skip:skip + n]], dtype=bool)


def cdf(g):
    return 0.5 * torch.special.erfc(-g / math.sqrt(2.0))


def activation(g, act):
    """(act(g), act'(g)) in 64 bits."""
    g = g.double()
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == "gelu":
        return g * cdf(g), cdf(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    return g.clamp(min=0), (g > 0).double()
