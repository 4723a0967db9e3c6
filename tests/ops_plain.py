"""The operators around the reduce in 64 bits, from their formulas, on the host.

Test infrastructure: numpy only, none of the package's code.  Inputs are
numpy arrays; results are float64.
"""

import math

import numpy as np

_ERF = np.vectorize(math.erf, otypes=[np.float64])
PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)


def philox4x32_10(counter, key):
    """The published generator on Python integers: four 32-bit words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = c[0] * PHILOX_M[0], c[2] * PHILOX_M[1]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + PHILOX_W[0]) & 0xFFFFFFFF, (k[1] + PHILOX_W[1]) & 0xFFFFFFFF]
    return c


def dropout_values(rows, cols, seed, offset):
    """16-bit value of every element."""
    u64 = np.uint64
    g = -(-cols // 8)
    c = [np.broadcast_to(np.arange(g, dtype=u64), (rows, g)),
         np.broadcast_to(np.arange(rows, dtype=u64)[:, None], (rows, g)),
         np.full((rows, g), offset & 0xFFFFFFFF, u64), np.full((rows, g), offset >> 32, u64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    m, h = u64(0xFFFFFFFF), u64(32)
    for _ in range(10):
        p0, p1 = c[0] * u64(PHILOX_M[0]), c[2] * u64(PHILOX_M[1])
        c = [(p1 >> h) ^ c[1] ^ u64(k[0]), p1 & m, (p0 >> h) ^ c[3] ^ u64(k[1]), p0 & m]
        k = [(k[0] + PHILOX_W[0]) & 0xFFFFFFFF, (k[1] + PHILOX_W[1]) & 0xFFFFFFFF]
    u = np.stack([x for w in c for x in (w & u64(0xFFFF), w >> u64(16))], axis=-1)
    return u.reshape(rows, 8 * g)[:, :cols].astype(np.int64)


def dropout_scale(rows, cols, p, seed, offset):
    """65536 / (65536 - T) where kept, 0 where dropped."""
    T = round(65536 * p)
    keep = dropout_values(rows, cols, seed, offset) >= T
    return np.where(keep, 65536.0 / max(65536 - T, 1), 0.0)


def dropout(x, scale):
    """A dropped element contributes 0 whatever it is."""
    return np.where(scale > 0, np.where(scale > 0, x, 0.0) * scale, 0.0)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, weight=None, dresidual=None):
    xh = (x - mean[:, None]) * rstd[:, None]
    q = dy if weight is None else dy * weight
    dx = rstd[:, None] * (q - q.mean(1, keepdims=True) - xh * (q * xh).mean(1, keepdims=True))
    if dresidual is not None:
        dx = dx + dresidual
    return dx, (dy * xh).sum(0), dy.sum(0)


def act(z, name):
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu":
        return 0.5 * z * (1 + _ERF(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + _ERF(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + z * s * (1 - s)
    return np.ones_like(z)
