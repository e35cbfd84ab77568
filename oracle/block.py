"""Reference of the operators around the attention in numpy float64, written out from their definitions:
rotary positions on a grid, layer norm, the generator of dropout, and the window softmax with dropout or as the
difference of two maps, each with its gradient.  Test infrastructure: shares no code with the library.
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------------------------

def rope(x, freqs, origin=None, amplitude=1.0, layout="half", inverse=False):
    """x [B, L.., heads, D]; freqs[a]: radians per position of axis a's pairs."""
    x = np.asarray(x, dtype=np.float64)
    n = x.ndim - 3
    origin = [0] * n if origin is None else origin
    y = x.copy()
    base = 0
    for a in range(n):
        f = np.asarray(freqs[a], dtype=np.float64)
        half = len(f)
        pos = np.array([float(origin[a] + i) for i in range(x.shape[1 + a])])
        theta = np.outer(pos, f) * (-1.0 if inverse else 1.0)
        shape = [1] * x.ndim
        shape[1 + a], shape[-1] = len(pos), half
        c, s = np.cos(theta).reshape(shape), np.sin(theta).reshape(shape)
        i = np.arange(half)
        lo, hi = (base + i, base + half + i) if layout == "half" else (base + 2 * i, base + 2 * i + 1)
        u, v = x[..., lo], x[..., hi]
        y[..., lo] = amplitude * (u * c - v * s)
        y[..., hi] = amplitude * (u * s + v * c)
        base += 2 * half
    return y


# ---------------------------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------------------------

def layernorm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[..., None]
    if w is not None:
        y = y * np.asarray(w, dtype=np.float64)
    if b is not None:
        y = y + np.asarray(b, dtype=np.float64)
    return y, mean, rstd


def layernorm_bwd(dy, x, w, mean, rstd):
    """(dx, dw, db) at the given statistics."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    mean, rstd = np.asarray(mean, dtype=np.float64)[..., None], np.asarray(rstd, dtype=np.float64)[..., None]
    h = (x - mean) * rstd
    g = dy if w is None else dy * np.asarray(w, dtype=np.float64)
    dx = rstd * (g - g.mean(-1, keepdims=True) - h * (g * h).mean(-1, keepdims=True))
    C = x.shape[-1]
    return dx, (dy * h).reshape(-1, C).sum(0), dy.reshape(-1, C).sum(0)


# ---------------------------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------------------------

def philox(counter, key, rounds):
    """Philox4x32 (Salmon et al., 2011) of counters [n, 4] under one key [2], in Python-exact integers."""
    c = [np.asarray(counter, dtype=np.uint64)[:, i].copy() for i in range(4)]
    k = [int(key[0]), int(key[1])]
    mask = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & mask,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def dropout_factor(n, p, seed, offset):
    """What dropout multiplies elements 0 .. n-1 by."""
    steps = int(np.floor((1.0 - p) * 65536 + 0.5))
    if steps == 65536:
        return np.ones(n)
    blocks = (n + 7) // 8
    i = np.arange(blocks, dtype=np.uint64)
    low, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    counter = np.stack([i & low, i >> shift, np.full(blocks, offset & 0xFFFFFFFF, np.uint64),
                        np.full(blocks, (offset >> 32) & 0xFFFFFFFF, np.uint64)], 1)
    words = philox(counter, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF), 7)
    fields = np.empty((blocks, 8), dtype=np.uint64)
    fields[:, 0::2] = words & np.uint64(0xFFFF)
    fields[:, 1::2] = words >> np.uint64(16)
    kept = fields.reshape(-1)[:n] < steps
    return np.where(kept, 65536.0 / steps if steps else 0.0, 0.0)


# ---------------------------------------------------------------------------------------------
# Window softmax with dropout, and the difference of two maps
# ---------------------------------------------------------------------------------------------

def softmax(x):
    """Over the last axis; a row of -inf alone gives zeros."""
    x = np.asarray(x, dtype=np.float64)
    m = x.max(-1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(invalid="ignore"):
        e = np.exp(x - m)
    t = e.sum(-1, keepdims=True)
    return e / np.where(t == 0, 1.0, t)


def softmax_dropout(x, factor):
    s = softmax(x)
    return np.where(factor == 0, 0.0, s * factor)


def softmax_dropout_bwd(x, dy, factor):
    s = softmax(x)
    g = np.where(factor == 0, 0.0, np.asarray(dy, dtype=np.float64) * factor)
    g = np.where(s == 0, 0.0, g)   # a place of weight zero takes no part
    return s * (g - (s * g).sum(-1, keepdims=True))


def diff_softmax(x1, x2, lam, factor):
    """lam: [heads] or [B, L.., heads]."""
    y = softmax(x1) - np.asarray(lam, dtype=np.float64)[..., None] * softmax(x2)
    return np.where(factor == 0, 0.0, y * factor)


def diff_softmax_bwd(x1, x2, lam, dy, factor):
    """(dx1, dx2, dlam)."""
    lam = np.asarray(lam, dtype=np.float64)
    dx1 = softmax_dropout_bwd(x1, dy, factor)
    dx2 = -lam[..., None] * softmax_dropout_bwd(x2, dy, factor)
    s2 = softmax(x2)
    g = np.where(factor == 0, 0.0, np.asarray(dy, dtype=np.float64) * factor)
    r2 = np.where(s2 == 0, 0.0, s2 * np.where(s2 == 0, 0.0, g)).sum(-1)
    return dx1, dx2, (-r2 if lam.ndim > 1 else -r2.reshape(-1, lam.shape[0]).sum(0))
