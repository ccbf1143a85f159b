"""fp64 causal linear attention with a decay per head, by its recurrence.
TEST INFRASTRUCTURE ONLY (see the package docstring).

    S_t = exp(g_h) S_{t-1} + k_t^T v_t,   o_t = scale q_t S_t

Sequences end at their ``lengths``; rows behind give zeros.  Gradients by the
recurrence run backwards, G_s = exp(g) G_{s+1} + scale q_s^T dO_s with the
gradient of the last state added at the last row:

    dq_t = scale S_t dO_t,  dk_s = G_s v_s,  dv_s = k_s G_s,  dS_0 = exp(g) G_0
"""
from __future__ import annotations

import numpy as np

from .attention import _f64


def _lengths(lengths, B, S):
    if lengths is None:
        return np.full(B, S)
    return np.clip(np.asarray(lengths, dtype=np.int64), 0, S)


def decay_attention(q, k, v, g, scale, state=None, lengths=None):
    """(o, state after the last row) of [B, H, S, D] inputs; rows behind a
    sequence's length may hold anything."""
    q, k, v, g = _f64(q), _f64(k), _f64(v), _f64(g)
    B, H, S, D = q.shape
    n = _lengths(lengths, B, S)
    lam = np.exp(g)[:, None, None]
    o = np.zeros_like(q)
    end = np.zeros((B, H, D, D)) if state is None else np.array(np.broadcast_to(_f64(state), (B, H, D, D)))
    for b in range(B):
        s = end[b].copy()
        for t in range(n[b]):
            s = lam * s + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * np.einsum("hd,hde->he", q[b, :, t], s)
        end[b] = s
    return o, end


def decay_attention_backward(q, k, v, do, g, scale, state=None, dstate=None, lengths=None):
    """(dq, dk, dv, dS_0)."""
    q, k, v, do, g = _f64(q), _f64(k), _f64(v), _f64(do), _f64(g)
    B, H, S, D = q.shape
    n = _lengths(lengths, B, S)
    lam = np.exp(g)[:, None, None]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    first = np.zeros((B, H, D, D)) if dstate is None else np.array(np.broadcast_to(_f64(dstate), (B, H, D, D)))
    for b in range(B):
        s = np.zeros((H, D, D)) if state is None else np.broadcast_to(_f64(state), (B, H, D, D))[b].copy()
        for t in range(n[b]):
            s = lam * s + k[b, :, t, :, None] * v[b, :, t, None, :]
            dq[b, :, t] = scale * np.einsum("hde,he->hd", s, do[b, :, t])
        s = first[b].copy()   # the loss's derivative by the state after row t
        for t in range(n[b] - 1, -1, -1):
            s = s + scale * q[b, :, t, :, None] * do[b, :, t, None, :]
            dk[b, :, t] = np.einsum("hde,he->hd", s, v[b, :, t])
            dv[b, :, t] = np.einsum("hd,hde->he", k[b, :, t], s)
            s = lam * s
        first[b] = s
    return dq, dk, dv, first
