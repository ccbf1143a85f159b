"""fp64 rotary positions and a cache of keys and values in pages.  TEST
INFRASTRUCTURE ONLY (see the package docstring)."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .attention import _f64

# pi to 50 digits, as a fraction
_PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


def rotary_cos_sin(positions, frequencies):
    """(cos, sin) [..., pairs] of position times frequency, the angle taken
    modulo 2 pi in exact arithmetic."""
    positions = np.asarray(positions)
    flat = positions.reshape(-1)
    two_pi = 2 * _PI
    f = [Fraction(float(x)) / two_pi for x in frequencies]          # turns a position
    known = {}
    for p in set(int(x) for x in flat):
        known[p] = [2 * math.pi * float(t - math.floor(t + Fraction(1, 2))) for t in (x * p for x in f)]
    angle = np.array([known[int(p)] for p in flat]).reshape(*positions.shape, len(f))
    return np.cos(angle), np.sin(angle)


def rotary(x, cos, sin, layout, amplitude=1.0, transposed=False):
    """x [..., S, D] turned; cos, sin broadcast to [..., S, pairs]."""
    y = _f64(x).copy()
    n = cos.shape[-1]
    i = np.arange(n)
    a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    s = -sin if transposed else sin
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a] = amplitude * (u * cos - w * s)
    y[..., b] = amplitude * (u * s + w * cos)
    return y


def _row(table, b, page, i):
    return int(table[b][i // page]), i % page


def paged_append(pool, rows, table, lengths, counts):
    """`pool` [pages, Hkv, page, D] with rows [B, Hkv, T, D] behind each
    request's lengths[b]."""
    out = np.array(pool, copy=True)
    for b in range(rows.shape[0]):
        for t in range(max(0, min(int(counts[b]), rows.shape[2]))):
            page, r = _row(table, b, pool.shape[2], max(0, int(lengths[b])) + t)
            out[page, :, r] = rows[b, :, t]
    return out


def paged_accept(pool, table, lengths, path, accepted):
    out = np.array(pool, copy=True)
    for b in range(len(lengths)):
        for i in range(int(accepted[b])):
            src, dst = (_row(table, b, pool.shape[2], int(lengths[b]) + x) for x in (int(path[b][i]), i))
            out[dst[0], :, dst[1]] = pool[src[0], :, src[1]]
    return out


def tree_attention(q, kp, vp, table, lengths, counts, tree, scale):
    """(o [B, H, T, D], lse [B, H, T], mean |v| under the softmax) of q [B, H, T,
    D] over pools [pages, Hkv, page, D].  tree: words [B][T] or None."""
    q, kp, vp = _f64(q), _f64(kp), _f64(vp)
    B, H, T, D = q.shape
    Hkv, page = kp.shape[1:3]
    o, a = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((B, H, T), -np.inf)
    for b in range(B):
        n, c = max(0, int(lengths[b])), max(0, min(int(counts[b]), T))
        if c == 0:
            continue
        at = np.arange(n + c)
        pages = np.asarray([int(x) for x in table[b]])[at // page]
        keys, values = (p[pages, :, at % page] for p in (kp, vp))       # [n + c, Hkv, D]
        for t in range(c):
            word = (1 << (t + 1)) - 1 if tree is None else int(tree[b][t]) % (1 << 64)
            sees = np.array([True] * n + [bool(word >> u & 1) for u in range(c)], dtype=bool)
            if not sees.any():
                continue
            for h in range(H):
                hk = h // (H // Hkv)
                s = scale * keys[sees, hk] @ q[b, h, t]
                m = s.max()
                p = np.exp(s - m)
                lse[b, h, t] = m + np.log(p.sum())
                o[b, h, t] = p @ values[sees, hk] / p.sum()
                a[b, h, t] = p @ np.abs(values[sees, hk]) / p.sum()
    return o, lse, a
