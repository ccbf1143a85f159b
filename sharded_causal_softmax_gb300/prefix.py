"""Decode attention of a batch that shares a long prefix
(``prefix_attn_decode`` of the C ABI).

The prefix's keys and values are kept, and read, once for the whole batch;
every request adds its own suffix cache.  The (o, lse) partials over pieces of
both are merged exactly by log-sum-exp rescaling, like the partials of
``ShardedCausalAttention``.  PyTorch supplies device memory and streams only.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import capi

def _sig(t):
    """What a call's checks look at besides the address."""
    return None if t is None else (t.dtype, t.device, t.shape, t.stride())


_DT = {torch.bfloat16: capi.SCA_BF16, torch.float32: capi.SCA_F32}


class SharedPrefixAttention:
    """Buffers and launches of one decode configuration: B requests of
    ``tokens`` newest tokens each (1, or a few verified together), H query
    heads on ``kv_heads`` key/value heads, at most ``prefix`` shared and
    ``suffix`` own keys (either may be 0).

    The outputs and the workspace belong to the plan: every call overwrites
    those of the call before, and calls in flight at once (other streams,
    captured graphs replayed side by side) need plans of their own.
    """

    def __init__(self, B, H, D, prefix, suffix, kv_heads=None, tokens=1, dtype=torch.bfloat16, scale=None,
                 device=None, algo=capi.SCA_ALGO_AUTO):
        if dtype not in _DT:
            raise ValueError(f"dtype {dtype}")
        if D not in (64, 128):
            raise ValueError(f"D={D}: only 64 and 128")
        Hkv = H if kv_heads is None else int(kv_heads)
        if B < 1 or H < 1 or Hkv < 1 or H % Hkv or B * H > 65535:
            raise ValueError(f"B={B}, H={H}, kv_heads={Hkv}: kv_heads must divide H, B*H be in [1, 65535]")
        if tokens < 1 or H // Hkv * tokens > 128:
            raise ValueError(f"{H // Hkv} heads a key/value head x {tokens} tokens: 1 to 128 query rows")
        if prefix < 0 or suffix < 0:
            raise ValueError(f"prefix={prefix}, suffix={suffix}")
        if algo == capi.SCA_ALGO_TC and dtype != torch.bfloat16:
            raise ValueError("the tensor-core kernel takes bf16 inputs only")
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        if dev.type != "cuda":
            raise ValueError(f"device {dev}: a CUDA device is needed")
        self.B, self.H, self.Hkv, self.T, self.D = B, H, Hkv, tokens, D
        self.prefix, self.suffix, self.dtype, self.device = prefix, suffix, dtype, dev
        self.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
        if not (math.isfinite(self.scale) and self.scale > 0):
            raise ValueError("scale must be finite and positive")
        self.algo = algo
        self._mult = 8 if dtype == torch.bfloat16 else 4
        self.o = torch.empty((B, H, tokens, D), dtype=dtype, device=dev)
        self.lse = torch.empty((B, H, tokens), dtype=torch.float32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._own = (self.o.data_ptr(), self.o.data_ptr() + self.o.numel() * self.o.element_size())
        self._seen = {}   # checked calls by their tensors' signatures
        with torch.cuda.device(dev):
            n = capi.prefix_attn_workspace(self._make_dims(H * tokens * D, prefix, suffix, (Hkv * prefix * D, D),
                                                           (Hkv * suffix * D, suffix * D, D)))
        self._ws = torch.empty(max(1, n // 4), dtype=torch.float32, device=dev)
        self._lib, self._call = capi.lib(), capi.Caller(dev)
        self._out_args = (self.o.data_ptr(), self.lse.data_ptr(), self._ws.data_ptr(), self._ws.numel() * 4,
                          self.status.data_ptr())

    def _make_dims(self, q_b, prefix, suffix, pv, sv):
        d = capi.sca_prefix_dims()
        d.B, d.H, d.Hkv, d.T, d.D = self.B, self.H, self.Hkv, self.T, self.D
        d.dtype, d.algo, d.scale = _DT[self.dtype], self.algo, self.scale
        d.q_b, d.prefix_len, d.suffix_cap = q_b, prefix, suffix
        d.prefix = capi.view(0, *pv)
        d.suffix = capi.view(*sv)
        return d

    def _pair(self, k, v, lead, most, what):
        """(rows, strides of the leading axes and of the rows) of a k, v pair, both of one layout."""
        if k is None or v is None:
            if k is not None or v is not None:
                raise ValueError(f"{what}: k and v go together")
            return 0, (0,) * len(lead) + (self.D,)
        rows = k.shape[-2] if k.dim() == len(lead) + 2 else -1
        if not 0 <= rows <= most:
            raise ValueError(f"{what}: {rows} rows, the plan takes up to {most}")
        shape = (*lead, rows, self.D)
        for t in (k, v):
            if t.dtype != self.dtype or t.device != self.device or tuple(t.shape) != shape:
                raise ValueError(f"{what}: expected {self.dtype} {shape} on {self.device}, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
        if k.stride() != v.stride():
            raise ValueError(f"{what}: k and v must have the same strides ({k.stride()}, {v.stride()})")
        st = list(k.stride())
        for i, n in enumerate(shape[:-1]):
            if n <= 1:   # a stride that no index is multiplied with may be anything
                st[i] = self.D if i == len(lead) else 0
        if (self.D > 1 and st[-1] != 1) or any(x % self._mult for x in st[:-1]) or st[-2] < self.D:
            raise ValueError(f"{what}: D must be contiguous, rows apart by at least D elements, and the strides "
                             f"multiples of 16 bytes (strides {k.stride()})")
        return rows, tuple(st[:-1])

    def decode(self, q, k_prefix, v_prefix, k_suffix, v_suffix, lengths):
        """(o [B, H, T, D], lse [B, H, T]) of the newest tokens.  k_prefix,
        v_prefix: [kv_heads, n, D] with n up to the plan's prefix, or None;
        k_suffix, v_suffix: [B, kv_heads, cap, D], of which request b uses the
        first lengths[b] rows (int32 [B] on the device), its T newest tokens'
        own the last among them, or None.  A newest token's value that is not
        finite shows, in its feature, in the tokens before it as well."""
        key = (_sig(q), _sig(k_prefix), _sig(v_prefix), _sig(k_suffix), _sig(v_suffix), _sig(lengths))
        entry = self._seen.get(key)
        if entry is None:
            entry = self._check(q, k_prefix, v_prefix, k_suffix, v_suffix, lengths)
            if len(self._seen) >= 64:
                self._seen.clear()
            self._seen[key] = entry
        _, ref, has_prefix, has_suffix = entry
        qp = q.data_ptr()
        ps = [k_prefix.data_ptr(), v_prefix.data_ptr()] if has_prefix else [None, None]
        ps += [k_suffix.data_ptr(), v_suffix.data_ptr(), lengths.data_ptr()] if has_suffix else [None, None, None]
        if (qp | (ps[0] or 0) | (ps[1] or 0) | (ps[2] or 0) | (ps[3] or 0)) & 15:
            raise ValueError("tensors must be 16-byte aligned")
        if self._own[0] <= qp < self._own[1]:
            raise ValueError("q lies in the plan's own output buffer")
        self._call(self._lib.prefix_attn_decode, ref, qp, *ps, *self._out_args)
        return self.o, self.lse

    def _check(self, q, k_prefix, v_prefix, k_suffix, v_suffix, lengths):
        """A call's sizes and strides; what it is to be made with."""
        shape = (self.B, self.H, self.T, self.D)
        if q.dtype != self.dtype or q.device != self.device or tuple(q.shape) != shape:
            raise ValueError(f"q: expected {self.dtype} {shape} on {self.device}, got {q.dtype} {tuple(q.shape)} on "
                             f"{q.device}")
        one = self.H * self.T * self.D
        q_b = q.stride(0) if self.B > 1 else one
        if not q[0].is_contiguous() or q_b % self._mult or q_b < one:
            raise ValueError(f"q: [H, T, D] must be contiguous and the batch stride at least {one} and a multiple of "
                             f"16 bytes (strides {q.stride()})")
        np, pv = self._pair(k_prefix, v_prefix, (self.Hkv,), self.prefix, "prefix")
        ns, sv = self._pair(k_suffix, v_suffix, (self.B, self.Hkv), self.suffix, "suffix")
        if ns and (lengths is None or lengths.dtype != torch.int32 or lengths.device != self.device or
                   tuple(lengths.shape) != (self.B,) or not lengths.is_contiguous()):
            raise ValueError(f"lengths: expected contiguous int32 ({self.B},) on {self.device}")
        d = self._make_dims(q_b, np, ns, pv, sv)
        return d, ctypes.byref(d), np > 0, ns > 0

    def read_status(self) -> int:
        """Synchronise and return the device status word (0 = OK; the
        tensor-core kernel records a timed-out wait there)."""
        return capi.sca_read_status(self.status.data_ptr(), torch.cuda.current_stream(self.device).cuda_stream)
