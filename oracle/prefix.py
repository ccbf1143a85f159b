"""fp64 decode attention over a shared prefix and each request's own suffix.
TEST INFRASTRUCTURE ONLY (see the package docstring)."""
from __future__ import annotations

import numpy as np

from .attention import _f64


def prefix_decode(q, kp, vp, ks, vs, lengths, scale):
    """(o [B, H, T, D], lse [B, H, T], mean |v| under the softmax) of q [B, H,
    T, D] over prefix [Hkv, n, D] and suffix [B, Hkv, cap, D] keys; token t
    sees suffix keys below lengths[b] - (T - 1 - t).  Either pair may be None."""
    q = _f64(q)
    B, H, T, D = q.shape
    Hkv = (kp if kp is not None else ks).shape[-3]
    o, a = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((B, H, T), -np.inf)
    for b in range(B):
        for h in range(H):
            hk = h // (H // Hkv)
            for t in range(T):
                keys, values = [], []
                if kp is not None:
                    keys.append(_f64(kp[hk]))
                    values.append(_f64(vp[hk]))
                if ks is not None:
                    n = int(np.clip(int(lengths[b]), 0, ks.shape[2])) - (T - 1 - t)
                    keys.append(_f64(ks[b, hk, :max(0, n)]))
                    values.append(_f64(vs[b, hk, :max(0, n)]))
                keys, values = np.concatenate(keys), np.concatenate(values)
                if len(keys) == 0:
                    continue
                s = scale * keys @ q[b, h, t]
                m = s.max()
                p = np.exp(s - m)
                lse[b, h, t] = m + np.log(p.sum())
                o[b, h, t] = p @ values / p.sum()
                a[b, h, t] = p @ np.abs(values) / p.sum()
    return o, lse, a
