"""Layer norm, dropout and the embedding in 64 bits, from their formulas, with
their gradients. Functions take and return NumPy arrays; nothing is shared with
the library.

Those named ``*_bound`` say how far a computation in fp32 may be from the 64-bit
result before its output is rounded to a shorter type: to first order, with each
operation off by at most U = 2^-24 of its result, and `depth` additions at most
between an element and the sum it is part of.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24
M32 = (1 << 32) - 1
# half a step, relative to the value, and half the smallest step
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}


def rounding(x, t):
    """The most that rounding x to type t moves it (the error of a bound's x
    inside is of second order)."""
    return np.abs(x) * HALF[t] + LEAST[t]


# ---- dropout --------------------------------------------------------------------

def philox4x32(counter, key, rounds):
    """Salmon et al. 2011: four words for one counter (4 words) and key (2)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & M32, (a >> 32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def random16(first, n, seed, offset):
    """16 random bits for each of the elements first .. first + n - 1."""
    g = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    m = np.uint64(M32)
    s = np.uint64(32)
    off = np.uint64(offset & ((1 << 64) - 1))
    c = [g & m, g >> s, np.full_like(g, off & m), np.full_like(g, off >> s)]
    k0, k1 = seed & M32, seed >> 32 & M32
    for _ in range(7):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k0), b & m, (a >> s) ^ c[3] ^ np.uint64(k1), a & m]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    w = np.stack(c, 1).astype(np.uint32).view(np.uint16)     # little endian: the lower half first
    at = first % 8
    return w.reshape(-1)[at:at + n]


def limit(p):
    return math.floor(p * 65536 + 0.5)


def factors(shape, p, seed, offset):
    """What each element is multiplied by: 0 or 1 / (1 - limit / 65536)."""
    t, n = limit(p), int(np.prod(shape))
    if t == 0:
        return np.ones(shape)
    if t == 65536:
        return np.zeros(shape)
    return ((random16(0, n, seed, offset) >= t) * (65536 / (65536 - t))).reshape(shape)


def dropped(x, f):
    """0 where the factor is, whatever x is there."""
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(f == 0, 0.0, x * f)


def dropout(x, f, residual=None):
    y = dropped(x, f)
    return y if residual is None else y + residual


def dropout_bound(x, f, residual=None):
    """The factor and the product are rounded, and the sum."""
    b = 2 * U * np.abs(dropped(x, f))
    return b if residual is None else b + U * np.abs(dropped(x, f) + residual)


# ---- layer norm -----------------------------------------------------------------

def layer_norm(z, w=None, b=None, eps=1e-5):
    """y, mean, rstd of rows z."""
    mean = z.mean(1, keepdims=True)
    d = z - mean
    rstd = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    y = d * rstd
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean, rstd


def layer_norm_bound(z, z_err, w, b, eps, depth):
    """Bounds of y, mean and rstd, for inputs that are z_err off."""
    y, mean, rstd = layer_norm(z, w, b, eps)
    d = np.abs(z - mean)
    var = (d * d).mean(1, keepdims=True)
    e_mean = z_err.mean(1, keepdims=True) + (depth + 2) * U * np.abs(z).mean(1, keepdims=True)
    e_d = z_err + e_mean + U * d
    # the mean's own error moves the variance in second order only, but is part of e_d here
    e_var = (2 * d * e_d + e_d ** 2).mean(1, keepdims=True) + (depth + 3) * U * var
    rel = 0.5 * e_var / (var + eps) + 4 * U
    e_n = e_d * rstd + d * rstd * (rel + U)
    e_y = e_n * (1.0 if w is None else np.abs(w)) + U * np.abs(y)
    return e_y, e_mean, rstd * rel


def layer_norm_backward(dy, h, mean, rstd, w=None, grad_h=None):
    """dh, dweight, dbias."""
    n = (h - mean) * rstd
    g = dy if w is None else dy * w
    dh = rstd * (g - g.mean(1, keepdims=True) - n * (g * n).mean(1, keepdims=True))
    if grad_h is not None:
        dh = dh + grad_h
    return dh, (dy * n).sum(0), dy.sum(0)


def layer_norm_backward_bound(dy, h, mean, rstd, w, grad_h, depth, rows_depth):
    n = np.abs((h - mean) * rstd)
    g = np.abs(dy) if w is None else np.abs(dy * w)
    m0, m1 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
    # n: 2 roundings; g: 1; its product with n: 4; the means: depth and the factor's 2
    e0, e1 = (depth + 3) * U * m0, (depth + 6) * U * m1
    e = rstd * (U * g + e0 + n * e1 + 2 * U * n * m1 + 3 * U * (g + m0 + n * m1))
    if grad_h is not None:
        e = e + U * (np.abs(grad_h) + rstd * (g + m0 + n * m1))
    return e, (rows_depth + 3) * U * (np.abs(dy) * n).sum(0), rows_depth * U * np.abs(dy).sum(0)


# ---- embedding ------------------------------------------------------------------

def embedding(tokens, table, scale=1.0, residual=None):
    t = np.asarray(tokens).reshape(-1)
    inside = (t >= 0) & (t < len(table))
    y = np.zeros((len(t), table.shape[1]))
    y[inside] = scale * table[t[inside]]
    return y if residual is None else y + residual


def embedding_bound(tokens, table, scale=1.0, residual=None):
    """scale and its product are rounded, and the sum."""
    y = np.abs(embedding(tokens, table, scale))
    b = 2 * U * y
    return b if residual is None else b + U * (y + np.abs(residual))


def embedding_backward(dy, tokens, vocab, scale=1.0):
    """The sums, place by place."""
    d = np.zeros((vocab, dy.shape[1]))
    for i, t in enumerate(np.asarray(tokens).reshape(-1)):
        if 0 <= t < vocab:
            d[t] += dy[i]
    return scale * d


def embedding_backward_bound(dy, tokens, vocab, scale=1.0):
    """m summands in any order: at most m roundings of the sum of magnitudes; the
    scale's two; adding to the old value is the output's rounding or one more."""
    t = np.asarray(tokens).reshape(-1)
    count = np.bincount(t[(t >= 0) & (t < vocab)], minlength=vocab)[:, None]
    return (count + 3) * U * embedding_backward(np.abs(dy), tokens, vocab, abs(scale))
