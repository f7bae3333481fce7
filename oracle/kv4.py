"""Float64 oracle of the 4-bit key/value cache (include/gbkv4.h), in numpy: the
format's quantisation with its float32 roundings, its byte layout, and attention
over rows taken from a paged cache.  Test infrastructure only."""

from __future__ import annotations

import numpy as np

GROUP = 64


def bf16_round(x):
    """float32 -> the nearest bfloat16 (ties to even), as float32.  Finite inputs."""
    w = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    w = (w + 0x7FFF + ((w >> 16) & 1)) & 0xFFFF0000
    return w.astype(np.uint32).view(np.float32).reshape(np.shape(x))


def quantise(x):
    """x [..., D] -> codes uint8 [..., D] (0 .. 15), s and b float32 [..., D / 64]."""
    g = np.asarray(x, np.float32).reshape(*np.shape(x)[:-1], np.shape(x)[-1] // GROUP, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    s = bf16_round((hi - lo) / np.float32(15))
    s = np.where(s < np.float32(2.0 ** -126), np.float32(0), s)
    b = bf16_round(lo + np.float32(8) * s)
    inv = np.divide(np.float32(1), s, out=np.zeros_like(s), where=s > 0)
    u = np.rint((g - b[..., None]) * inv[..., None]) + np.float32(8)
    return np.clip(u, 0, 15).astype(np.uint8).reshape(np.shape(x)), s, b


def pack(codes):
    """codes [..., D] -> bytes [..., D / 2]: 32-bit words [8][groups], word (i, g) with
    the values 8 i .. 8 i + 7 of group g, the first in its lowest 4 bits."""
    D = codes.shape[-1]
    out = np.zeros((*codes.shape[:-1], D // 2), np.uint8)
    n_groups = D // GROUP
    for d in range(D):
        g, i, n = d // GROUP, d % GROUP // 8, d % 8
        out[..., (i * n_groups + g) * 4 + n // 2] |= codes[..., d] << (4 * (n % 2))
    return out


def unpack(packed):
    D = 2 * packed.shape[-1]
    out = np.zeros((*packed.shape[:-1], D), np.uint8)
    n_groups = D // GROUP
    for d in range(D):
        g, i, n = d // GROUP, d % GROUP // 8, d % 8
        out[..., d] = (packed[..., (i * n_groups + g) * 4 + n // 2] >> (4 * (n % 2))) & 15
    return out


def parts(codes, s, b):
    """s (u - 8) and b, each spread over [..., D], in float64."""
    s64, b64 = (np.repeat(np.asarray(t, np.float64), GROUP, -1) for t in (s, b))
    return s64 * (codes.astype(np.float64) - 8), b64


def rows(codes, scale, table_row, page, length):
    """One sequence's rows of a cache: codes [pages, H, page, D / 2], scale [pages, H,
    page, D / 64, 2] float -> (u [H, length, D], s, b [H, length, D / 64])."""
    ids = np.asarray(table_row[: -(-length // page)], dtype=np.int64)
    c = codes[ids].transpose(1, 0, 2, 3).reshape(codes.shape[1], len(ids) * page, codes.shape[3])[:, :length]
    sc = scale[ids].transpose(1, 0, 2, 3, 4).reshape(scale.shape[1], len(ids) * page, scale.shape[3], 2)[:, :length]
    return unpack(c), sc[..., 0], sc[..., 1]


def attend(q, k_parts, v_parts, k_s, scale, causal):
    """q [Hq, t, D] over one sequence's n rows; k_parts and v_parts are parts() of the
    rows [Hkv, n, D], k_s the keys' s [Hkv, n, D / 64].  Query i sits at position n - t + i.

    Returns float64 o [Hq, t, D], lse [Hq, t] and what error bounds are made of:
    A = sum_j p_j (|s (u - 8)| + |b|), R = sum_j p_j |s (u - 8)| (both [Hq, t, D]),
    W = the largest scale * sum_d |q_d| (16 s + |b|) over the keys a row sees [Hq, t]."""
    Hq, t, D = q.shape
    Hkv, n, _ = k_parts[0].shape
    o, A, R = (np.zeros((Hq, t, D)) for _ in range(3))
    lse, W = np.full((Hq, t), -np.inf), np.zeros((Hq, t))
    size = 16 * np.repeat(np.asarray(k_s, np.float64), GROUP, -1) + np.abs(k_parts[1])
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        k, v = k_parts[0][kv] + k_parts[1][kv], v_parts[0][kv] + v_parts[1][kv]
        for i in range(t):
            last = max(0, n - t + i + 1) if causal else (n if n - t + i >= 0 else 0)
            if last == 0:
                continue
            x = scale * (k[:last] @ q[h, i])
            m = x.max()
            e = np.exp(x - m)
            lse[h, i] = m + np.log(e.sum())
            p = e / e.sum()
            o[h, i] = p @ v[:last]
            R[h, i] = p @ np.abs(v_parts[0][kv][:last])
            A[h, i] = R[h, i] + p @ np.abs(v_parts[1][kv][:last])
            W[h, i] = abs(scale) * (size[kv, :last] @ np.abs(q[h, i])).max()
    return o, lse, A, R, W
