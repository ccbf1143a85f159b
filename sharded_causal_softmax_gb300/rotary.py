"""Rotary positions of queries and keys (``rotary_apply`` of the C ABI).

    y_a = m (x_a cos(p f_i) - x_b sin(p f_i)),   y_b = m (x_a sin(p f_i) + x_b cos(p f_i))

for the pairs (a, b) of a row's first ``rotary_dim`` features at position p;
the features behind them stay.  ``RotaryAngles`` holds the frequencies and the
layout, ``RotaryPositions`` the buffers and launches of one configuration;
``ShardedCausalAttention`` and ``PagedKVCache`` take angles too and turn what
they are given.  PyTorch supplies device memory and streams only.
"""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import torch

from . import capi

_DT = {torch.bfloat16: capi.SCA_BF16, torch.float32: capi.SCA_F32}

# 2 pi to 128 bits behind the point
_TWO_PI = Fraction(2138057168129933495719360746323741566601, 1 << 128)


def _sig(t):
    """What a call's checks look at besides the address."""
    return None if t is None else (t.dtype, t.device, t.shape, t.stride())


def cuda_device(device):
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if dev.type != "cuda":
        raise ValueError(f"device {dev}: a CUDA device is needed")
    return dev


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None):
    """(frequencies in radians a position, one a pair, in 64 bits; amplitude).

    f_i = base^(-2 i / rotary_dim), and with ``scaling`` for contexts s times
    as long as the trained ones
      ("linear", s)   f_i / s: positions moved closer together;
      ("base", s)     base s^(rotary_dim / (rotary_dim - 2)): the lowest
                      frequency divided by s, the highest kept;
      ("ramp", s, trained[, low, high])   f_i where a pair turns more than
                      ``high`` (32) times over the ``trained`` positions,
                      f_i / s where less than ``low`` (1) times, a line between
                      them in the number of turns; amplitude 0.1 ln s + 1.
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim={rotary_dim}: even and at least 2")
    if not (math.isfinite(base) and base > 0):
        raise ValueError(f"base={base}")
    kind, amplitude = None, 1.0
    if scaling is not None:
        kind, s, *more = scaling
        if kind not in ("linear", "base", "ramp") or len(more) not in ({"ramp": (1, 3)}.get(kind, (0,))):
            raise ValueError(f"scaling {scaling!r}")
        if not (math.isfinite(s) and s >= 1):
            raise ValueError(f"scaling {scaling!r}: the factor must be at least 1")
    if kind == "base" and rotary_dim > 2:
        base = base * s ** (rotary_dim / (rotary_dim - 2))
    f = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if kind == "linear":
        f = [x / s for x in f]
    if kind == "ramp":
        trained, low, high = (*more, 1.0, 32.0) if len(more) == 1 else more
        if not (trained > 0 and 0 <= low < high):
            raise ValueError(f"scaling {scaling!r}: needs trained > 0 and 0 <= low < high")
        keep = [min(1.0, max(0.0, (trained * x / (2 * math.pi) - low) / (high - low))) for x in f]
        f = [x * (g + (1.0 - g) / s) for x, g in zip(f, keep)]
        amplitude = 0.1 * math.log(s) + 1.0
    return f, amplitude


class RotaryAngles:
    """Which angles a position means: the frequencies of ``rotary_dim / 2``
    pairs and their layout, "half" (pairs (i, i + rotary_dim / 2)) or
    "interleaved" (pairs (2 i, 2 i + 1)).  ``base`` and ``scaling`` as in
    ``rotary_frequencies``; or ``frequencies`` (radians a position, finite) and
    ``amplitude`` themselves.

    ``turns`` holds the frequencies on the device as 64-bit fractions of a turn,
    so that the angles of any position are exact.  It does not change after
    this and may be shared by any number of plans.
    """

    def __init__(self, rotary_dim, base=10000.0, layout="half", scaling=None, frequencies=None, amplitude=None,
                 device=None):
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout {layout!r}")
        if frequencies is None:
            f, a = rotary_frequencies(rotary_dim, base, scaling)
        else:
            if scaling is not None:
                raise ValueError("frequencies are taken as they are: no scaling beside them")
            f, a = torch.as_tensor(frequencies, dtype=torch.float64).reshape(-1).tolist(), 1.0
            if rotary_dim < 2 or rotary_dim % 2 or len(f) != rotary_dim // 2 or not all(math.isfinite(x) for x in f):
                raise ValueError(f"frequencies must hold rotary_dim / 2 = {rotary_dim / 2:g} finite numbers")
        a = a if amplitude is None else float(amplitude)
        if not math.isfinite(a):
            raise ValueError("amplitude is not finite")
        self.device = cuda_device(device)
        self.rotary_dim, self.layout, self.frequencies, self.amplitude = rotary_dim, layout, f, a
        words = [round(Fraction(x) / _TWO_PI * (1 << 64)) % (1 << 64) for x in f]
        words = [w - (1 << 64) if w >> 63 else w for w in words]
        self.turns = torch.tensor(words, dtype=torch.int64).to(self.device)


def check_positions(positions, B, rows, device, what="positions"):
    """The batch stride of int32 [B, rows] or [rows] positions."""
    if positions.dtype != torch.int32 or positions.device != device or \
            tuple(positions.shape) not in ((B, rows), (rows,)) or (rows > 1 and positions.stride(-1) != 1):
        raise ValueError(f"{what}: expected int32 ({B}, {rows}) or ({rows},) on {device}, rows contiguous, got "
                         f"{positions.dtype} {tuple(positions.shape)} on {positions.device}")
    return positions.stride(0) if positions.dim() == 2 and B > 1 else 0


class RotaryPositions:
    """Buffers and launches of one configuration: queries of H heads and keys
    of ``kv_heads`` (H if not given), of at most ``S`` rows.

    Inputs are [B, heads, rows, D] tensors of ``dtype`` (bf16 or fp32) on the
    plan's device, D contiguous, any other strides.  The outputs belong to the
    plan: every call overwrites those of the call before, so that none of them
    may be an input, and calls in flight at once (other streams, captured
    graphs replayed side by side) need plans of their own.
    """

    def __init__(self, B, H, S, D, angles, kv_heads=None, dtype=torch.bfloat16, backward=False, device=None):
        if dtype not in _DT:
            raise ValueError(f"dtype {dtype}")
        Hkv = H if kv_heads is None else int(kv_heads)
        if B < 1 or H < 1 or Hkv < 1 or H + Hkv > 65535 or not 1 <= S < 1 << 31 or B * S >= 1 << 36:
            raise ValueError(f"B={B}, H={H}, kv_heads={Hkv}, S={S}: need positive sizes, H + kv_heads <= 65535")
        if D < 2 or D % 2 or D > 1024:
            raise ValueError(f"D={D}: even, up to 1024")
        if angles.rotary_dim > D:
            raise ValueError(f"rotary_dim={angles.rotary_dim} of D={D}")
        self.device = cuda_device(device if device is not None else angles.device)
        if angles.device != self.device:
            raise ValueError(f"the angles are on {angles.device}, the plan on {self.device}")
        self.B, self.H, self.Hkv, self.S, self.D, self.dtype = B, H, Hkv, S, D, dtype
        self.angles, self.backward_enabled = angles, backward
        nq, nk = B * H * S * D, B * Hkv * S * D
        self._own = torch.empty((2 if backward else 1) * (nq + nk), dtype=dtype, device=self.device)
        parts = self._own.split([nq, nk] * (2 if backward else 1))
        self._q, self._k = parts[:2]
        if backward:
            self._dq, self._dk = parts[2:]
        lo = self._own.data_ptr()
        self._range = (lo, lo + self._own.numel() * self._own.element_size())
        self._seen = {}        # checked calls by their tensors' signatures
        self._held = None      # rows and positions of the last forward
        self._lib, self._call = capi.lib(), capi.Caller(self.device)

    def _strides(self, t, heads, rows, what):
        shape = (self.B, heads, rows, self.D)
        if t.dtype != self.dtype or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{what}: expected {self.dtype} {shape} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        st = t.stride()
        if st[-1] != 1:
            raise ValueError(f"{what}: D must be contiguous (strides {st})")
        return tuple(0 if n == 1 else s for s, n in zip(st[:3], shape))

    def _run(self, q, k, positions, transposed, qo, ko):
        key = (_sig(q), _sig(k), _sig(positions), transposed)
        entry = self._seen.get(key)
        if entry is None:
            rows = q.shape[2] if q.dim() == 4 else 0
            if not 1 <= rows <= self.S:
                raise ValueError(f"{rows} rows: the plan takes 1 to {self.S}")
            d = capi.sca_rotary_dims()
            d.B, d.H, d.Hkv, d.D, d.S, d.dtype = self.B, self.H, self.Hkv, self.D, rows, _DT[self.dtype]
            d.rotary_dim, d.interleaved = self.angles.rotary_dim, int(self.angles.layout == "interleaved")
            d.amplitude, d.transposed = self.angles.amplitude, int(transposed)
            what = ("dq", "dk") if transposed else ("q", "k")
            d.q = capi.view(*self._strides(q, self.H, rows, what[0]))
            d.k = capi.view(*self._strides(k, self.Hkv, rows, what[1]))
            if positions is not None:
                d.pos_b = check_positions(positions, self.B, rows, self.device)
            n = rows * self.D
            d.qo, d.ko = capi.view(self.H * n, n, self.D), capi.view(self.Hkv * n, n, self.D)
            out = tuple(t[:self.B * h * n].view(self.B, h, rows, self.D) for t, h in ((qo, self.H), (ko, self.Hkv)))
            if len(self._seen) >= 64:
                self._seen.clear()
            entry = self._seen[key] = (d, ctypes.byref(d), out, out[0].data_ptr(), out[1].data_ptr())
        _, ref, out, qo, ko = entry
        qp, kp = q.data_ptr(), k.data_ptr()
        lo, hi = self._range
        if lo <= qp < hi or lo <= kp < hi:
            raise ValueError("an input lies in one of the plan's own output buffers")
        self._call(self._lib.rotary_apply, ref, qp, kp, self.angles.turns.data_ptr(),
                   None if positions is None else positions.data_ptr(), qo, ko)
        return out

    def forward(self, q, k, positions=None):
        """(q, k) turned to their positions: int32 [B, rows] or [rows] on the
        device, any values; the rows' indices if not given."""
        self._held = None
        out = self._run(q, k, positions, False, self._q, self._k)
        if self.backward_enabled:
            self._held = (q.shape[2], positions)
        return out

    def backward(self, dq, dk):
        """(dq, dk) by the last forward's inputs, from those by its results.
        The positions are the last forward's (kept by reference)."""
        if not self.backward_enabled:
            raise RuntimeError("plan built without backward=True")
        if self._held is None:
            raise RuntimeError("backward before forward")
        rows, positions = self._held
        if dq.dim() != 4 or dq.shape[2] != rows:
            raise ValueError(f"dq: {tuple(dq.shape)}, the last forward had {rows} rows")
        return self._run(dq, dk, positions, True, self._dq, self._dk)
