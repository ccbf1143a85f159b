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


def _sig(t):
    """What a call's checks look at besides the address."""
    return t.dtype, t.device, t.shape, t.stride()


class DecayLinearAttention:
    """Buffers and launches of one configuration; ``S`` is the most rows a
    call may bring.  ``log_decay``: [H] fp32 values <= 0 (the log of each
    head's decay, a constant of the model), checked here once.

    Inputs are [B, H, rows, D] tensors of ``dtype`` (bf16 or fp32) on the
    plan's device, D contiguous and the other strides multiples of 16 bytes;
    outputs have the same dtype, states are fp32 [B, H, D, D].  The outputs
    and the workspace belong to the plan: every call overwrites those of the
    call before, so that none of them may be an input (a state may be handed
    on), and calls in flight at once (other streams, captured graphs replayed
    side by side) need plans of their own.
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
        if dev.type != "cuda":
            raise ValueError(f"device {dev}: a CUDA device is needed")
        g = torch.as_tensor(log_decay, dtype=torch.float32).detach()
        if tuple(g.shape) != (H,) or not bool((g <= 0).all()):
            raise ValueError(f"log_decay must hold {H} values <= 0 (logs of decays in [0, 1])")
        self.B, self.H, self.S, self.D, self.dtype, self.device = B, H, S, D, dtype, dev
        self.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
        if not math.isfinite(self.scale):
            raise ValueError("scale is not finite")
        self.algo, self.backward_enabled = algo, backward
        self.log_decay = g.to(dev, copy=True).contiguous()
        # every output that a caller could hand back as an input by mistake lies in one buffer
        n, n1 = B * H * S * D, B * H * D
        own = torch.empty((4 if backward else 1) * n + n1, dtype=dtype, device=dev)
        self._o1 = own[:n1].view(B, H, D)
        self._o, *grads = own[n1:].view(-1, B, H, S, D)
        if backward:
            self._dq, self._dk, self._dv = grads
            self.dstate = torch.empty((B, H, D, D), dtype=torch.float32, device=dev)
        self._own = (own.data_ptr(), own.data_ptr() + own.numel() * own.element_size())
        self.state = torch.empty((B, H, D, D), dtype=torch.float32, device=dev)
        # an fp32 plan's states have a shape that inputs may have as well
        self._own_states = None
        if dtype == torch.float32:
            a, b = (t.data_ptr() for t in (self.state, self.dstate if backward else self.state))
            n1 = self.state.numel() * 4
            self._own_states = (a, a + n1, b, b + n1)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._mult = 8 if dtype == torch.bfloat16 else 4
        self._seen = {}        # checked calls by their tensors' signatures
        self._held = None      # what the last forward ran on
        with torch.cuda.device(dev):
            n = capi.decay_attn_workspace(self._make_dims(S, *([(H * S * D, S * D, D)] * 3)), int(backward))
        self._ws = torch.empty(max(1, n // 4), dtype=torch.float32, device=dev)
        self._lib, self._call = capi.lib(), capi.Caller(dev)
        self._g_ptr, self._state_ptr, self._o1_ptr = (t.data_ptr() for t in (self.log_decay, self.state, self._o1))
        self._ws_args = (self._ws.data_ptr(), self._ws.numel() * 4)
        self._status_ptr = self.status.data_ptr()

    # ------------------------------------------------------------ helpers

    def _make_dims(self, S, q, k, v):
        d = capi.sca_decay_dims()
        d.B, d.H, d.D, d.S = self.B, self.H, self.D, S
        d.dtype, d.algo, d.scale = _DT[self.dtype], self.algo, self.scale
        d.q, d.k, d.v = capi.view(*q), capi.view(*k), capi.view(*v)
        d.o = capi.view(self.H * S * self.D, S * self.D, self.D)
        return d

    def _strides(self, t, rows, what):
        """(batch, head, row) strides of an input; rows = 0: a single token's, without a row axis."""
        shape = (self.B, self.H, rows, self.D) if rows else (self.B, self.H, self.D)
        if t.dtype != self.dtype or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{what}: expected {self.dtype} {shape} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        st = t.stride()
        m, D = self._mult, self.D
        # a stride that no index is multiplied with may be anything
        b = st[0] if self.B > 1 else 0
        h = st[1] if self.H > 1 else 0
        s = st[2] if rows > 1 else D
        if st[-1] != 1 or b % m or h % m or s % m or s < D:
            raise ValueError(f"{what}: D must be contiguous, rows apart by at least D elements, and the other strides "
                             f"multiples of 16 bytes (strides {st})")
        return b, h, s

    def _addresses(self, *ts):
        lo, hi = self._own
        ps = []
        for t in ts:
            p = t.data_ptr()
            if p & 15 or lo <= p < hi:
                raise ValueError("tensors must be 16-byte aligned" if p & 15 else
                                 "an input lies in one of the plan's own output buffers")
            ps.append(p)
        if self._own_states:
            a, b, c, d = self._own_states
            for p in ps:
                if a <= p < b or c <= p < d:
                    raise ValueError("an input lies in one of the plan's own state buffers")
        return ps

    def _keep(self, key, entry):
        if len(self._seen) >= 64:
            self._seen.clear()
        self._seen[key] = entry
        return entry

    def _state(self, t, what):
        """The batch stride; 0 (``expand``) shares one state."""
        shape = (self.B, self.H, self.D, self.D)
        if t.dtype != torch.float32 or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{what}: expected float32 {shape} on {self.device}, got {t.dtype} {tuple(t.shape)} on "
                             f"{t.device}")
        one = self.H * self.D * self.D
        if tuple(t.stride()[1:]) != (self.D * self.D, self.D, 1) and not (
                self.H == 1 and tuple(t.stride()[2:]) == (self.D, 1)):
            raise ValueError(f"{what}: each sequence's states must be contiguous (strides {t.stride()})")
        b = t.stride(0) if self.B > 1 else one
        if b % 4 or (b and b < one):
            raise ValueError(f"{what}: batch stride {b} must be 0 or at least {one}")
        return b

    def _lengths(self, lengths):
        if lengths.dtype != torch.int32 or lengths.device != self.device or tuple(lengths.shape) != (self.B,) or \
                not lengths.is_contiguous():
            raise ValueError(f"lengths: expected contiguous int32 ({self.B},) on {self.device}")

    # -------------------------------------------------------------- calls

    def forward(self, q, k, v, state=None, lengths=None):
        """(o, state after each sequence's last row).  ``state``: the states
        to start from ([B, H, D, D]; ``expand`` one to share it), zero if not
        given.  ``lengths``: int32 [B]; rows behind them are not read and give
        zeros.  A plan without backward may be handed its own ``state`` back;
        one with backward keeps the inputs by reference and needs ``state``
        to stay what it was.  A value that is not finite shows, in its
        feature, in rows before it as well: those of its chunk of 128 (fp32
        arithmetic: 64)."""
        key = (_sig(q), _sig(k), _sig(v), None if state is None else _sig(state),
               None if lengths is None else _sig(lengths))
        entry = self._seen.get(key)
        if entry is None:
            rows = q.shape[2] if q.dim() == 4 else 0
            if not 1 <= rows <= self.S:
                raise ValueError(f"{rows} rows: the plan takes 1 to {self.S}")
            d = self._make_dims(rows, self._strides(q, rows, "q"), self._strides(k, rows, "k"),
                                self._strides(v, rows, "v"))
            if lengths is not None:
                self._lengths(lengths)
            entry = self._keep(key, (d, ctypes.byref(d), 0 if state is None else self._state(state, "state"),
                                     self._rows(self._o, rows)))
        d, ref, sb, o = entry
        qp, kp, vp = self._addresses(q, k, v)
        sp = None if state is None else state.data_ptr()
        if self.backward_enabled and state is not None and \
                state.untyped_storage().data_ptr() == self.state.untyped_storage().data_ptr():
            raise ValueError("a plan with backward cannot start from its own state buffer: pass a copy")
        lp = None if lengths is None else lengths.data_ptr()
        self._held = None
        self._call(self._lib.decay_attn_fwd, ref, qp, kp, vp, self._g_ptr, lp, sp, sb, o.data_ptr(), self._state_ptr,
                   *self._ws_args, self._status_ptr)
        if self.backward_enabled:
            self._held = (d, ref, q, k, v, state, sb, lengths)
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
        d, ref, q, k, v, state, sb, lengths = self._held
        key = (d.S, _sig(do), None if dstate is None else _sig(dstate))
        entry = self._seen.get(key)
        if entry is None:
            dov = capi.view(*self._strides(do, d.S, "do"))
            entry = self._keep(key, (dov, ctypes.byref(dov), 0 if dstate is None else self._state(dstate, "dstate"),
                                     [self._rows(t, d.S) for t in (self._dq, self._dk, self._dv)]))
        _, dov, db, grads = entry
        qp, kp, vp, op = self._addresses(q, k, v, do)
        if dstate is not None and dstate.untyped_storage().data_ptr() == self.dstate.untyped_storage().data_ptr():
            raise ValueError("dstate lies in the plan's own dstate buffer: pass a copy")
        self._call(self._lib.decay_attn_bwd, ref, qp, kp, vp, op, dov, self._g_ptr,
                   None if lengths is None else lengths.data_ptr(), None if state is None else state.data_ptr(), sb,
                   None if dstate is None else dstate.data_ptr(), db, grads[0].data_ptr(), grads[1].data_ptr(),
                   grads[2].data_ptr(), None if state is None else self.dstate.data_ptr(), *self._ws_args, 1,
                   self._status_ptr)
        return (*grads, None if state is None else self.dstate)

    def step(self, q, k, v, state):
        """o [B, H, D] of one token of every sequence; ``state`` (a prompt's,
        or the last step's) is updated in place.  q, k, v: [B, H, D]."""
        key = (_sig(q), _sig(k), _sig(v), _sig(state))
        entry = self._seen.get(key)
        if entry is None:
            d = self._make_dims(1, self._strides(q, 0, "q"), self._strides(k, 0, "k"), self._strides(v, 0, "v"))
            sb = self._state(state, "state")
            if sb == 0:
                raise ValueError("state: every sequence needs a state of its own")
            entry = self._keep(key, (d, ctypes.byref(d), sb))
        _, ref, sb = entry
        qp, kp, vp = self._addresses(q, k, v)
        sp = state.data_ptr()
        if sp & 15 or self._own[0] <= sp < self._own[1]:
            raise ValueError("the state must be 16-byte aligned" if sp & 15 else
                             "the state lies in one of the plan's own output buffers")
        self._call(self._lib.decay_attn_step, ref, qp, kp, vp, self._g_ptr, sp, sb, self._o1_ptr)
        return self._o1

    def read_status(self) -> int:
        """Synchronise and return the device status word (0 = OK; the
        tensor-core kernels record a timed-out wait there)."""
        return capi.sca_read_status(self._status_ptr, torch.cuda.current_stream(self.device).cuda_stream)

    def _rows(self, buf, rows):
        n = self.B * self.H * rows * self.D   # a call of fewer rows than the plan's: the buffer's first part
        return buf.reshape(-1)[:n].reshape(self.B, self.H, rows, self.D)
