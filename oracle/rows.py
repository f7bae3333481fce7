"""Oracle for dropout, LayerNorm's backward pass and the embedding table: the plain
definitions in whole numbers and float64.

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``).

The dropout's bits are Philox4x32's (Salmon, Moraes, Dror, Shaw: "Parallel random
numbers: as easy as 1, 2, 3", 2011), in Python's unsigned 64-bit numpy arithmetic.
"""

from __future__ import annotations

import numpy as np

from .ln import ln_residual

M32 = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key, rounds: int):
    """Four 32-bit words (as uint64 arrays) for a counter of four and a key of two 32-bit words."""
    x = [np.asarray(c, dtype=np.uint64) for c in counter]
    k = [int(v) for v in key]
    for _ in range(rounds):
        p0, p1 = np.uint64(0xD2511F53) * x[0], np.uint64(0xCD9E8D57) * x[2]
        x = [(p1 >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), p1 & M32,
             (p0 >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), p0 & M32]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return x


def dropout_bits(rows, cols: int, seed: int, offset: int):
    """The 16 bits of every element, [rows, cols]; rows: how many, or an array of row numbers."""
    r = np.arange(rows, dtype=np.uint64) if np.isscalar(rows) else np.asarray(rows, dtype=np.uint64)
    groups = np.arange((cols + 7) // 8, dtype=np.uint64)
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    shape = (len(r), len(groups))
    one = np.ones(shape, dtype=np.uint64)
    words = philox4x32([groups[None, :] * one, r[:, None] * one, np.uint64(offset % 2 ** 32) * one,
                        np.uint64(offset >> 32) * one], (seed % 2 ** 32, seed >> 32), 7)
    u = np.empty((*shape, 8), dtype=np.uint64)
    for e in range(8):
        u[..., e] = (words[e // 2] >> np.uint64(16 * (e % 2))) & np.uint64(0xFFFF)
    return u.reshape(len(r), -1)[:, :cols]


def dropout(x, p: float, seed: int, offset: int, rows=None):
    """D(x) for x [rows, cols]; rows: the row numbers where x holds some rows of a larger tensor."""
    x = np.asarray(x, dtype=np.float64)
    t = int(np.floor(65536 * p + 0.5))
    u = dropout_bits(x.shape[0] if rows is None else rows, x.shape[1], seed, offset)
    out = np.zeros_like(x)
    keep = u >= t
    if t < 65536:
        out[keep] = x[keep] * (65536.0 / (65536 - t))
    return out


def ln_dropout_residual(x, residual, gamma, beta, eps, p, seed, offset):
    """(y, h, mean, rstd) of LayerNorm(D(x) + residual)."""
    return ln_residual(dropout(x, p, seed, offset), residual, gamma, beta, eps)


def ln_bwd(dy, h, mean, rstd, gamma=None, dh=None):
    """(dr, dgamma, dbeta)."""
    dy, h = np.asarray(dy, dtype=np.float64), np.asarray(h, dtype=np.float64)
    mean, rstd = (np.asarray(v, dtype=np.float64)[:, None] for v in (mean, rstd))
    xh = (h - mean) * rstd
    g = dy if gamma is None else dy * np.asarray(gamma, dtype=np.float64)
    n = dy.shape[1]
    dr = rstd * (g - g.sum(1, keepdims=True) / n - xh * ((g * xh).sum(1, keepdims=True) / n))
    if dh is not None:
        dr = dr + np.asarray(dh, dtype=np.float64)
    return dr, (dy * xh).sum(0), dy.sum(0)


def embedding(weight, ids, scale: float = 1.0):
    """scale * weight[ids]; 0 for an id outside the table."""
    weight, ids = np.asarray(weight, dtype=np.float64), np.asarray(ids)
    ok = (ids >= 0) & (ids < weight.shape[0])
    out = np.zeros((*ids.shape, weight.shape[1]))
    out[ok] = scale * weight[ids[ok]]
    return out


def embedding_bwd(dy, ids, vocab: int, scale: float = 1.0, padding_id=None):
    """The table's gradient, and the sum of the magnitudes that each of its elements is made of."""
    dy, ids = np.asarray(dy, dtype=np.float64).reshape(-1, np.shape(dy)[-1]), np.asarray(ids).reshape(-1)
    dw, size = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < vocab and v != padding_id:
            dw[v] += scale * dy[i]
            size[v] += abs(scale) * np.abs(dy[i])
    return dw, size
