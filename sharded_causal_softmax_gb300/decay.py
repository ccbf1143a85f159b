"""Causal linear attention with a decay per head: prompts, training and
single tokens (``decay_attn_*`` of the C ABI).

    S_t = exp(g_h) S_{t-1} + k_t^T v_t,      o_t = scale * q_t S_t

The recurrence of linear attention sequence parallelism ("Effiziente
Parallelisierung linearer Aufmerksamkeitssequenzen fuer skalierbare
Sprachmodelle") with an exponential decay.  The state is handed in and out:
a context shard is one ``forward`` from the state that the shard before it
returned, a batch of prompts can start from one shared prefix's state, and
``step`` goes on from a prompt's.  PyTorch supplies device memory and streams
only.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import capi

_DT = {torch.bfloat16: capi.SCA_BF16, torch.float32: capi.SCA_F32}


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


class DecayLinearAttention:
    """Buffers and launches of one configuration; ``S`` is the most rows a
    call may bring.  ``log_decay``: [H] fp32 values <= 0 (the log of each
    head's decay, a constant of the model), checked here once.

    Inputs are [B, H, rows, D] tensors of ``dtype`` (bf16 or fp32) on the
    plan's device, D contiguous and the other strides multiples of 16 bytes;
    outputs have the same dtype, states are fp32 [B, H, D, D].  The outputs
    and the workspace belong to the plan: every call overwrites those of the
    call before, and calls in flight at once (other streams, captured graphs
    replayed side by side) need plans of their own.
    """

    def __init__(self, B, H, S, D, log_decay, dtype=torch.bfloat16, scale=None, backward=False, device=None,
                 algo=capi.SCA_ALGO_AUTO):
        if dtype not in _DT:
            raise ValueError(f"dtype {dtype}")
        if D not in (64, 128):
            raise ValueError(f"D={D}: only 64 and 128")
        if B < 1 or H < 1 or B * H > 65535 or not 1 <= S < 1 << 24:
            raise ValueError(f"B={B}, H={H}, S={S}: need B*H in [1, 65535] and S in [1, 2^24)")
        if algo == capi.SCA_ALGO_TC and dtype != torch.bfloat16:
            raise ValueError("the tensor-core kernels take bf16 inputs only")
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        g = torch.as_tensor(log_decay, dtype=torch.float32).detach()
        if tuple(g.shape) != (H,) or not bool((g <= 0).all()):
            raise ValueError(f"log_decay must hold {H} values <= 0 (logs of decays in [0, 1])")
        self.B, self.H, self.S, self.D, self.dtype, self.device = B, H, S, D, dtype, dev
        self.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
        if not math.isfinite(self.scale):
            raise ValueError("scale is not finite")
        self.algo, self.backward_enabled = algo, backward
        self.log_decay = g.to(dev, copy=True).contiguous()
        z = lambda *shape, dt=dtype: torch.empty(shape, dtype=dt, device=dev)
        self._o = z(B, H, S, D)
        self.state = z(B, H, D, D, dt=torch.float32)
        self._o1 = z(B, H, D)
        if backward:
            self._dq, self._dk, self._dv = z(B, H, S, D), z(B, H, S, D), z(B, H, S, D)
            self.dstate = z(B, H, D, D, dt=torch.float32)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._mult = 8 if dtype == torch.bfloat16 else 4
        self._buffers = [t.untyped_storage().data_ptr() for t in
                         [self._o, self._o1] + ([self._dq, self._dk, self._dv] if backward else [])]
        self._dims = {}        # by rows and strides
        self._held = None      # what the last forward ran on
        with torch.cuda.device(dev):
            n = capi.decay_attn_workspace(self._make_dims(S, *([(H * S * D, S * D, D)] * 3)), int(backward))
        self._ws = torch.empty(max(1, n // 4), dtype=torch.float32, device=dev)

    # ------------------------------------------------------------ helpers

    def _make_dims(self, S, q, k, v):
        d = capi.sca_decay_dims()
        d.B, d.H, d.D, d.S = self.B, self.H, self.D, S
        d.dtype, d.algo, d.scale = _DT[self.dtype], self.algo, self.scale
        d.q, d.k, d.v = capi.view(*q), capi.view(*k), capi.view(*v)
        d.o = capi.view(self.H * S * self.D, S * self.D, self.D)
        return d

    def _strides(self, t, rows, what):
        shape = (self.B, self.H, rows, self.D)
        if t.dtype != self.dtype or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{what}: expected {self.dtype} {shape} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        st = t.stride()
        m, D = self._mult, self.D
        # a stride that no index is multiplied with may be anything
        b = st[0] if self.B > 1 else 0
        h = st[1] if self.H > 1 else 0
        s = st[2] if rows > 1 else D
        if st[3] != 1 or b % m or h % m or s % m or s < D or t.data_ptr() % 16:
            raise ValueError(f"{what}: D must be contiguous, rows apart by at least D elements, and the base and the "
                             f"other strides multiples of 16 bytes (strides {st})")
        if t.untyped_storage().data_ptr() in self._buffers:
            raise ValueError(f"{what} lies in one of the plan's own output buffers")
        return b, h, s

    def _state(self, t, what):
        """(pointer, batch stride); a stride of 0 (``expand``) shares one state."""
        shape = (self.B, self.H, self.D, self.D)
        if t.dtype != torch.float32 or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{what}: expected float32 {shape} on {self.device}, got {t.dtype} {tuple(t.shape)} on "
                             f"{t.device}")
        one = self.H * self.D * self.D
        if tuple(t.stride()[1:]) != (self.D * self.D, self.D, 1) and not (
                self.H == 1 and tuple(t.stride()[2:]) == (self.D, 1)) or t.data_ptr() % 16:
            raise ValueError(f"{what}: each sequence's states must be contiguous and 16-byte aligned "
                             f"(strides {t.stride()})")
        b = t.stride(0) if self.B > 1 else one
        if b % 4 or (b and b < one):
            raise ValueError(f"{what}: batch stride {b} must be 0 or at least {one}")
        return t.data_ptr(), b

    def _lengths(self, lengths):
        if lengths is None:
            return None
        if lengths.dtype != torch.int32 or lengths.device != self.device or tuple(lengths.shape) != (self.B,) or \
                not lengths.is_contiguous():
            raise ValueError(f"lengths: expected contiguous int32 ({self.B},) on {self.device}")
        return lengths.data_ptr()

    # -------------------------------------------------------------- calls

    def forward(self, q, k, v, state=None, lengths=None):
        """(o, state after each sequence's last row).  ``state``: the states
        to start from ([B, H, D, D]; ``expand`` one to share it), zero if not
        given.  ``lengths``: int32 [B]; rows behind them are not read and give
        zeros.  A plan without backward may be handed its own ``state`` back;
        one with backward keeps the inputs by reference and needs ``state``
        to stay what it was."""
        rows = q.shape[2] if q.dim() == 4 else 0
        if not 1 <= rows <= self.S:
            raise ValueError(f"{rows} rows: the plan takes 1 to {self.S}")
        views = (self._strides(q, rows, "q"), self._strides(k, rows, "k"), self._strides(v, rows, "v"))
        sp, sb = (None, 0) if state is None else self._state(state, "state")
        if self.backward_enabled and state is not None and \
                state.untyped_storage().data_ptr() == self.state.untyped_storage().data_ptr():
            raise ValueError("a plan with backward cannot start from its own state buffer: pass a copy")
        lp = self._lengths(lengths)
        with torch.cuda.device(self.device):
            d = self._dims.get((rows, views))
            if d is None:
                if len(self._dims) > 64:
                    self._dims.clear()
                d = self._dims[(rows, views)] = self._make_dims(rows, *views)
            st = torch.cuda.current_stream(self.device).cuda_stream
            o = self._o if rows == self.S else self._rows(self._o, rows)
            self._held = None
            capi.decay_attn_fwd(d, q.data_ptr(), k.data_ptr(), v.data_ptr(), self.log_decay.data_ptr(), lp, sp, sb,
                                o.data_ptr(), self.state.data_ptr(), self._ws.data_ptr(), self._ws.numel() * 4,
                                self.status.data_ptr(), st)
        if self.backward_enabled:
            self._held = (d, q, k, v, state, sp, sb, lengths, lp)
        return o, self.state

    def backward(self, do, dstate=None):
        """(dq, dk, dv, dstate0) of the last forward's inputs, from the
        gradients of its two results (``dstate`` zero if not given).
        dstate0, the gradient of the states started from (None if there were
        none), is [B, H, D, D] also where the batch shared one: that one's
        gradient is their sum."""
        if not self.backward_enabled:
            raise RuntimeError("plan built without backward=True")
        if self._held is None:
            raise RuntimeError("backward before forward")
        d, q, k, v, state, sp, sb, lengths, lp = self._held
        rows = d.S
        dov = capi.view(*self._strides(do, rows, "do"))
        dp, db = (None, 0) if dstate is None else self._state(dstate, "dstate")
        if dstate is not None and dstate.untyped_storage().data_ptr() == self.dstate.untyped_storage().data_ptr():
            raise ValueError("dstate lies in the plan's own dstate buffer: pass a copy")
        grads = [t if rows == self.S else self._rows(t, rows) for t in (self._dq, self._dk, self._dv)]
        with torch.cuda.device(self.device):
            st = torch.cuda.current_stream(self.device).cuda_stream
            capi.decay_attn_bwd(d, q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), dov,
                                self.log_decay.data_ptr(), lp, sp, sb, dp, db, grads[0].data_ptr(),
                                grads[1].data_ptr(), grads[2].data_ptr(), None if state is None else self.dstate.data_ptr(),
                                self._ws.data_ptr(), self._ws.numel() * 4, 1,
                                self.status.data_ptr(), st)
        return (*grads, None if state is None else self.dstate)

    def step(self, q, k, v, state):
        """o [B, H, D] of one token of every sequence; ``state`` (a prompt's,
        or the last step's) is updated in place.  q, k, v: [B, H, D]."""
        shape = (self.B, self.H, self.D)
        views = []
        for t, what in ((q, "q"), (k, "k"), (v, "v")):
            if t.dtype != self.dtype or t.device != self.device or tuple(t.shape) != shape:
                raise ValueError(f"{what}: expected {self.dtype} {shape} on {self.device}, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
            b, h, s = t.stride()
            b, h = b if self.B > 1 else 0, h if self.H > 1 else 0
            if s != 1 or b % self._mult or h % self._mult or t.data_ptr() % 16:
                raise ValueError(f"{what}: D must be contiguous, the base and the other strides multiples of 16 "
                                 f"bytes (strides {t.stride()})")
            if t.untyped_storage().data_ptr() in self._buffers:
                raise ValueError(f"{what} lies in one of the plan's own output buffers")
            views.append((b, h, self.D))
        sp, sb = self._state(state, "state")
        if sb == 0:
            raise ValueError("state: every sequence needs a state of its own")
        key = (0, *views)
        with torch.cuda.device(self.device):
            d = self._dims.get(key)
            if d is None:
                if len(self._dims) > 64:
                    self._dims.clear()
                d = self._dims[key] = self._make_dims(1, *views)
            st = torch.cuda.current_stream(self.device).cuda_stream
            capi.decay_attn_step(d, q.data_ptr(), k.data_ptr(), v.data_ptr(), self.log_decay.data_ptr(), sp, sb,
                                 self._o1.data_ptr(), st)
        return self._o1

    def read_status(self) -> int:
        """Synchronise and return the device status word (0 = OK; the
        tensor-core kernels record a timed-out wait there)."""
        return capi.sca_read_status(self.status.data_ptr(), torch.cuda.current_stream(self.device).cuda_stream)

    def _rows(self, buf, rows):
        n = self.B * self.H * rows * self.D
        return buf.reshape(-1)[:n].reshape(self.B, self.H, rows, self.D)
