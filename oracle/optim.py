"""The optimizer step behind a synchronisation, in 64 bits: the global gradient
norm, AdamW, and the 8-bit state format, from their formulas. Every function
takes and returns NumPy arrays; nothing is shared with the library.

With a step's outputs come bounds: how far an fp32 computation with one rounding
per operation (each off by at most U = 2^-24 of its result) may be from them.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24
BLOCK = 64
M32, M64 = (1 << 32) - 1, (1 << 64) - 1


def norm(grads, grad_scale=1.0):
    """sqrt of the exactly rounded sum of squares of all elements (fp64)."""
    total = 0.0
    for g in grads:
        g = np.asarray(g, dtype=np.float64).ravel()
        if not np.isfinite(g).all():
            return math.nan if np.isnan(g).any() else math.inf
        total = math.fsum([total, math.fsum((g * g).tolist())])
    return abs(grad_scale) * math.sqrt(total)


def clip_coef(n, max_norm):
    return max_norm / n if n > max_norm else 1.0


def adamw(w, g, m, v, *, t, lr, beta1, beta2, eps, weight_decay, gscale):
    """One step (number t) on fp64 arrays. Returns (w, m, v, r) and the bounds
    of their fp32 counterparts, in units of U and to first order:
      m  the gradient's term takes 4 roundings (its factor, the product, 1 -
         beta1, the product) and the sum one, the old m's term 2 and the sum;
      v  the gradient's term 2 * 2 + 1 + 2 and the sum, the old v's (with its
         square, for roots) 3 and the sum; r half of that and its own, 5;
      w  old w: its factor, the product, the last difference, 3; the update: m's
         bound, r's 5, 2 for its factor and product, 2 for eps and the sum, the
         quotient, the rate, the product and the last difference, 13 in all.
    """
    with np.errstate(all="ignore"):
        g = g * gscale
        a, b = beta1 * m, (1 - beta1) * g
        v = beta2 * v + (1 - beta2) * g * g
        r = np.sqrt(v)
        rate = lr / (1 - beta1 ** t)
        den = r / math.sqrt(1 - beta2 ** t) + eps
        m = a + b
        new = w * (1 - lr * weight_decay) - m / den * rate
        bm = 5 * U * (np.abs(a) + np.abs(b))
        bw = U * 3 * np.abs(w) + rate / den * (bm + 13 * U * np.abs(m))
    return (new, m, v, r), (bw, bm, 8 * U * v, 5 * U * r)


# ---- 8-bit states ------------------------------------------------------------------

def _code_values():
    out = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        if c & 127 == 127:
            x = math.nan
        out.append(-x if c & 128 else x)
    return np.array(out)


CODES = _code_values()


def scales_of(x):
    """The e8m0 byte of each block of 64: the smallest s >= 1 with
    max|x| <= 448 * 2^(s - 127), over the finite elements."""
    n = x.size
    a = np.zeros(-(-n // BLOCK) * BLOCK)
    a[:n] = np.where(np.isfinite(x), np.abs(x), 0.0)
    top = a.reshape(-1, BLOCK).max(1)
    s = np.ones(top.size, dtype=np.int64)
    for i, y in enumerate(top):
        if y > 0:
            s[i] = max(1, math.frexp(y / 448.0)[1] + 127 - (math.frexp(y / 448.0)[0] == 0.5))
    return s


def decode(codes, scales):
    """Values of uint8 codes under uint8 scales."""
    f = np.ldexp(1.0, scales.astype(np.int64) - 127)
    return CODES[codes] * np.repeat(f, BLOCK)[:codes.size]


def encode_levels(x, scales, u16, root):
    """Where |x| / scale falls between two neighbouring code values: the lower
    value, the next one up, and the exact position in steps with u / 65536
    added (it rounds up from 1 on)."""
    y = np.abs(x) / np.repeat(np.ldexp(1.0, scales - 127), BLOCK)[:x.size]
    e = np.maximum(np.frexp(y)[1] - 1, -6)
    q = np.ldexp(1.0, e - 3)
    low = np.floor(y / q)
    pos = y / q - low + u16 / 65536.0
    lo, hi = low * q, (low + 1) * q
    if root:
        lo = np.where(y > 0, np.maximum(lo, 2.0 ** -9), lo)
        hi = np.where(y > 0, np.maximum(hi, 2.0 ** -9), hi)
    return lo, hi, pos


def random16(seed, t, index):
    """The 16 random bits for m and for r of the elements at ``index`` (uint64;
    every variable's first element lies on a multiple of 64)."""
    k = (seed + t * 0xA3B1956C7E4D2F89) & M64
    k ^= k >> 32
    k = k * 0xD6C7F2A94B1E8653 & M64
    k ^= k >> 29
    k = k * 0x9E6B3F85C2D4A717 & M64
    k ^= k >> 32
    k0, k1 = np.uint64(k & M32), np.uint64(k >> 32)
    m = np.uint64(M32)
    sh = lambda x, b: x >> np.uint64(b)  # noqa: E731
    i = index.astype(np.uint64)
    gi = sh(i, 2)
    with np.errstate(over="ignore"):
        h = ((gi & m) * np.uint64(0x9C8E5A6D) + sh(gi, 32) * np.uint64(0x7F4A3C15) + k0) & m
        h = ((h ^ sh(h, 15)) * np.uint64(0x85D3B2A7)) & m
        h = ((h ^ sh(h, 13) ^ k1) * np.uint64(0xC5A7E36B)) & m
        h ^= sh(h, 16)
        x = (h + (i & np.uint64(3)) * np.uint64(0x6D2B4E95)) & m
        x = ((x ^ sh(x, 16)) * np.uint64(0xB5297A4D)) & m
        x ^= sh(x, 15)
    return sh(x, 16).astype(np.int64), (x & np.uint64(0xFFFF)).astype(np.int64)


def bases(numels):
    """Index of each variable's first element in the random bits' numbering."""
    out, at = [], 0
    for n in numels:
        out.append(at)
        at += -(-n // BLOCK) * BLOCK
    return out
