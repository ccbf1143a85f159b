"""A cache of keys and values in pages and the attention of newest tokens over
it (``paged_kv_append``, ``paged_tree_attend``, ``paged_kv_accept`` of the C
ABI).

A request's rows lie in pages of a pool that all requests share, found through
its table of page numbers.  A step of decoding is
``append`` (the new rows, turned to their positions, behind those that are
there) and ``attend`` (each new token over the request's rows: one token, a
piece of a prompt, or the nodes of a tree of drafted tokens, each of which sees
its ancestors); of drafted tokens ``accept`` then keeps the path that was right.
The table, the lengths and the pool are the caller's.  PyTorch supplies device
memory and streams only.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import capi
from .rotary import check_positions, cuda_device

_DT = {torch.bfloat16: capi.SCA_BF16, torch.float32: capi.SCA_F32}


def _sig(t):
    """What a call's checks look at besides the address."""
    return None if t is None else (t.dtype, t.device, t.shape, t.stride())


def _ptr(t):
    return None if t is None else t.data_ptr()


class PagedKVCache:
    """A pool of ``pages`` pages of ``page`` rows (16, 32, ... 1024) for
    ``kv_heads`` heads: ``k`` and ``v``, [pages, kv_heads, page, D] of ``dtype``
    (bf16 or fp32).  ``pools``: (k, v) views of the caller's instead of new
    ones, both of one layout, D contiguous and the other strides multiples of
    16 bytes (one layer of a pool that holds all layers; rows before heads).
    With ``angles`` the keys (and queries) of an append are turned to their
    positions; without, they are copied.

    Request b's row i is row i % page of page table[b, i // page] (int32 [B, n]
    on the device).  ``lengths`` (int32 [B]): the rows that are there before a
    call; ``counts`` (int32 [B]): how many of a call's rows are the request's,
    the others are padding.  Rows behind a table's end or on a page outside the
    pool are neither written nor used (``read_status`` then returns
    SCA_ERR_RANGE).  Requests may share pages that none of them writes.
    """

    def __init__(self, pages, kv_heads, D, page=64, dtype=torch.bfloat16, angles=None, pools=None, device=None):
        if dtype not in _DT:
            raise ValueError(f"dtype {dtype}")
        if page not in (16, 32, 64, 128, 256, 512, 1024):
            raise ValueError(f"page={page}: 16, 32, ... 1024 rows")
        mult = 8 if dtype == torch.bfloat16 else 4
        if not 1 <= pages < 1 << 31 or not 1 <= kv_heads <= 65535 or not mult <= D <= 1024 or D % mult:
            raise ValueError(f"pages={pages}, kv_heads={kv_heads}, D={D}: need positive sizes and D a multiple of 16 "
                             "bytes, up to 1024")
        if device is None and pools is not None:
            device = pools[0].device
        self.device = cuda_device(device)
        if angles is not None and (angles.device != self.device or angles.rotary_dim > D):
            raise ValueError(f"angles of {angles.rotary_dim} features on {angles.device}: the cache has D={D} on "
                             f"{self.device}")
        self.pages, self.Hkv, self.D, self.page, self.dtype, self.angles = pages, kv_heads, D, page, dtype, angles
        shape = (pages, kv_heads, page, D)
        if pools is None:
            self.k, self.v = (torch.empty(shape, dtype=dtype, device=self.device) for _ in range(2))
        else:
            self.k, self.v = pools
            for t in pools:
                if t.dtype != dtype or t.device != self.device or tuple(t.shape) != shape:
                    raise ValueError(f"pools: expected {dtype} {shape} on {self.device}, got {t.dtype} "
                                     f"{tuple(t.shape)} on {t.device}")
            st = self.k.stride()
            if st != self.v.stride() or st[-1] != 1 or any(s % mult for s in st[:-1]) or st[2] < D:
                raise ValueError(f"pools: one layout, D contiguous, strides multiples of 16 bytes ({st}, "
                                 f"{self.v.stride()})")
            if (self.k.data_ptr() | self.v.data_ptr()) & 15:
                raise ValueError("pools must be 16-byte aligned")
        st = self.k.stride()
        self._pool = tuple(0 if n == 1 else s for s, n in zip(st[:2], shape)) + (st[2],)
        self._kp, self._vp = self.k.data_ptr(), self.v.data_ptr()
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._status_ptr = self.status.data_ptr()
        self._turns = None if angles is None else angles.turns.data_ptr()
        self._seen = {}
        self._lib, self._call = capi.lib(), capi.Caller(self.device)

    # ------------------------------------------------------------ helpers

    def make_dims(self, B, T, table_shape, table_b):
        d = capi.sca_paged_dims()
        d.B, d.H, d.Hkv, d.T, d.D, d.dtype = B, self.Hkv, self.Hkv, T, self.D, _DT[self.dtype]
        d.page, d.pages, d.table_n, d.table_b = self.page, self.pages, table_shape, table_b
        d.pool, d.scale = capi.view(*self._pool), 1.0
        if self.angles is not None:
            d.rotary_dim, d.amplitude = self.angles.rotary_dim, self.angles.amplitude
            d.interleaved = int(self.angles.layout == "interleaved")
        return d

    def check_table(self, table, B):
        """(entries, batch stride) of a table."""
        if table.dtype != torch.int32 or table.device != self.device or table.dim() != 2 or table.shape[0] != B or \
                table.shape[1] < 1 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError(f"table: expected int32 ({B}, n) on {self.device}, entries contiguous, got {table.dtype} "
                             f"{tuple(table.shape)} on {table.device}")
        return table.shape[1], table.stride(0) if B > 1 else 0

    def check_ints(self, t, B, what):
        if t.dtype != torch.int32 or t.device != self.device or tuple(t.shape) != (B,) or not t.is_contiguous():
            raise ValueError(f"{what}: expected contiguous int32 ({B},) on {self.device}")

    def rows_view(self, t, B, heads, rows, what):
        shape = (B, heads, rows, self.D)
        if t.dtype != self.dtype or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{what}: expected {self.dtype} {shape} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        if t.stride(-1) != 1:
            raise ValueError(f"{what}: D must be contiguous (strides {t.stride()})")
        return capi.view(*(0 if n == 1 else s for s, n in zip(t.stride()[:3], shape)))

    def keep(self, key, entry):
        if len(self._seen) >= 64:
            self._seen.clear()
        self._seen[key] = entry
        return entry

    # -------------------------------------------------------------- calls

    def append(self, k, v, table, lengths, counts=None, positions=None):
        """Writes rows t < counts[b] (all, if not given) of k and v [B,
        kv_heads, rows, D] behind the lengths[b] rows of request b, the keys
        turned to positions (absolute, int32 [B, rows] or [rows]; lengths[b] + t
        if not given).  The lengths stay as they are: the rows count once the
        caller says so (or ``accept`` does).  k and v that lie in the pools are
        refused; two requests must not write one page."""
        self._append(None, k, v, table, lengths, counts, positions, None)

    def _append(self, q, k, v, table, lengths, counts, positions, q_out):
        key = (_sig(q), _sig(k), _sig(v), _sig(table), _sig(lengths), _sig(counts), _sig(positions))
        entry = self._seen.get(key)
        if entry is None:
            if k.dim() != 4 or k.shape[0] < 1 or k.shape[2] < 1:
                raise ValueError(f"k: expected [B, {self.Hkv}, rows, {self.D}], got {tuple(k.shape)}")
            B, rows = k.shape[0], k.shape[2]
            d = self.make_dims(B, rows, *self.check_table(table, B))
            d.k, d.v = self.rows_view(k, B, self.Hkv, rows, "k"), self.rows_view(v, B, self.Hkv, rows, "v")
            if q is not None:
                d.H = q.shape[1]
                d.q = self.rows_view(q, B, d.H, rows, "q")
            self.check_ints(lengths, B, "lengths")
            if counts is not None:
                self.check_ints(counts, B, "counts")
            if positions is not None:
                d.pos_b = check_positions(positions, B, rows, self.device)
            entry = self.keep(key, (d, ctypes.byref(d)))
        self._call(self._lib.paged_kv_append, entry[1], _ptr(q), k.data_ptr(), v.data_ptr(), table.data_ptr(),
                   lengths.data_ptr(), _ptr(counts), _ptr(positions), self._turns, self._kp, self._vp, q_out,
                   self._status_ptr)

    def read_status(self) -> int:
        """Synchronise and return the device status word (0 = OK, SCA_ERR_RANGE
        after a row without a place or a path that does not rise)."""
        return capi.sca_read_status(self._status_ptr, torch.cuda.current_stream(self.device).cuda_stream)


class PagedTreeAttention:
    """Buffers and launches of the steps of B requests over a ``cache`` (D 64
    or 128): ``tokens`` newest tokens a call, H query heads, tables of at most
    ``keys`` rows.

    The outputs and the workspace belong to the plan: every call overwrites
    those of the call before, and calls in flight at once (other streams,
    captured graphs replayed side by side) need plans of their own.  The
    workspace holds counters that each call leaves as it found them: zeroed
    when the plan is made, which its first call waits for on whatever stream it
    is (a first call that is captured does not: synchronise before), and to be
    zeroed again, by a plan made anew, after SCA_ERR_TIMEOUT.
    """

    def __init__(self, cache, B, H, tokens=1, keys=None, scale=None, algo=capi.SCA_ALGO_AUTO):
        Hkv, D, dev = cache.Hkv, cache.D, cache.device
        if B < 1 or H < 1 or H % Hkv or B * H > 65535:
            raise ValueError(f"B={B}, H={H}, kv_heads={Hkv}: kv_heads must divide H, B*H be in [1, 65535]")
        if tokens < 1 or H // Hkv * tokens > 65536:
            raise ValueError(f"{H // Hkv} heads a key/value head x {tokens} tokens: 1 to 65536 query rows")
        if D not in (64, 128):
            raise ValueError(f"D={D}: only 64 and 128")
        if algo == capi.SCA_ALGO_TC and cache.dtype != torch.bfloat16:
            raise ValueError("the tensor-core kernel takes bf16 inputs only")
        keys = cache.pages * cache.page if keys is None else int(keys)
        if keys < 1:
            raise ValueError(f"keys={keys}")
        self.cache, self.B, self.H, self.T, self.device = cache, B, H, tokens, dev
        cache._call.wait()   # (its status is this plan's too)
        self.entries = min(-(-keys // cache.page), ((1 << 31) - (1 << 20)) // cache.page - 1)
        self.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
        if not (math.isfinite(self.scale) and self.scale > 0):
            raise ValueError("scale must be finite and positive")
        self.algo, self._mult = algo, 8 if cache.dtype == torch.bfloat16 else 4
        self.q, self.o = (torch.empty((B, H, tokens, D), dtype=cache.dtype, device=dev) for _ in range(2))
        self.lse = torch.empty((B, H, tokens), dtype=torch.float32, device=dev)
        self.lengths = torch.empty((B,), dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._own = tuple((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in (self.q, self.o))
        self._seen = {}
        with torch.cuda.device(dev):
            n = capi.paged_tree_workspace(self._make_dims(self.entries, self.entries, H * tokens * D))
        # zeroed once: the counters in it return to zero at the end of every call
        self._ws = torch.zeros(max(1, n // 4), dtype=torch.float32, device=dev)
        self._lib, self._call = capi.lib(), capi.Caller(dev)
        self._out_args = (self.o.data_ptr(), self.lse.data_ptr(), self._ws.data_ptr(), self._ws.numel() * 4,
                          self.status.data_ptr())
        self._q_ptr, self._lengths_ptr = self.q.data_ptr(), self.lengths.data_ptr()

    def _make_dims(self, entries, table_b, q_b):
        d = self.cache.make_dims(self.B, self.T, entries, table_b)
        d.H, d.algo, d.scale = self.H, self.algo, self.scale
        d.q.b = q_b
        return d

    def _table(self, table):
        n, b = self.cache.check_table(table, self.B)
        if n > self.entries:
            raise ValueError(f"table: {n} entries, the plan takes up to {self.entries}")
        return n, b

    def append(self, q, k, v, table, lengths, counts=None, positions=None):
        """``PagedKVCache.append`` of the calls' ``tokens`` rows, and the
        queries q [B, H, tokens, D] turned to the same positions (zeros for
        padding), which ``attend`` takes.  Positions are absolute: drafted
        tokens at depths in a tree have lengths[:, None] + depths."""
        if tuple(q.shape) != (self.B, self.H, self.T, self.cache.D):
            raise ValueError(f"q: expected {(self.B, self.H, self.T, self.cache.D)}, got {tuple(q.shape)}")
        if self._own[0][0] <= q.data_ptr() < self._own[0][1]:
            raise ValueError("q lies in the plan's own output buffer")
        self.cache._append(q, k, v, table, lengths, counts, positions, self._q_ptr)
        return self.q

    def attend(self, q, table, lengths, counts=None, tree=None):
        """(o [B, H, tokens, D], lse [B, H, tokens]) of the newest tokens, whose
        own rows follow lengths[b] in the cache.  ``tree``: int64 [B, tokens] or
        [tokens], bit u of word t says that token t sees token u (its ancestors
        and itself; at most 64 tokens); not given: it sees those up to itself.
        Padding and rows that see nothing give 0 and -inf.  A newest token's
        value that is not finite shows, in its feature, in tokens that do not
        see it as well."""
        key = (_sig(q), _sig(table), _sig(lengths), _sig(counts), _sig(tree))
        entry = self._seen.get(key)
        if entry is None:
            entry = self._check(q, table, lengths, counts, tree)
            if len(self._seen) >= 64:
                self._seen.clear()
            self._seen[key] = entry
        qp = q.data_ptr()
        if qp & 15:
            raise ValueError("q must be 16-byte aligned")
        if self._own[1][0] <= qp < self._own[1][1]:
            raise ValueError("q lies in the plan's own output buffer")
        c = self.cache
        self._call(self._lib.paged_tree_attend, entry[1], qp, c._kp, c._vp, table.data_ptr(), lengths.data_ptr(),
                   _ptr(counts), _ptr(tree), *self._out_args)
        return self.o, self.lse

    def _check(self, q, table, lengths, counts, tree):
        B, H, T, D = shape = (self.B, self.H, self.T, self.cache.D)
        if q.dtype != self.cache.dtype or q.device != self.device or tuple(q.shape) != shape:
            raise ValueError(f"q: expected {self.cache.dtype} {shape} on {self.device}, got {q.dtype} "
                             f"{tuple(q.shape)} on {q.device}")
        one = H * T * D
        q_b = q.stride(0) if B > 1 else one
        if not q[0].is_contiguous() or q_b % self._mult or q_b < one:
            raise ValueError(f"q: [H, tokens, D] must be contiguous and the batch stride at least {one} and a multiple "
                             f"of 16 bytes (strides {q.stride()})")
        d = self._make_dims(*self._table(table), q_b)
        self.cache.check_ints(lengths, B, "lengths")
        if counts is not None:
            self.cache.check_ints(counts, B, "counts")
        if tree is not None:
            if T > 64:
                raise ValueError(f"a tree of {T} tokens: at most 64")
            if tree.dtype != torch.int64 or tree.device != self.device or tuple(tree.shape) not in ((B, T), (T,)) or \
                    (T > 1 and tree.stride(-1) != 1):
                raise ValueError(f"tree: expected int64 ({B}, {T}) or ({T},) on {self.device}, words contiguous")
            d.tree_b = tree.stride(0) if tree.dim() == 2 and B > 1 else 0
        return d, ctypes.byref(d)

    def accept(self, table, lengths, path, accepted, out=None):
        """Keeps the first accepted[b] nodes of path[b] (int32 [B, tokens], node
        numbers that rise) of the drafted tokens: their rows move up behind the
        lengths[b] rows that were there.  Returns the new lengths, in ``out``
        (which may be ``lengths``) or a buffer of the plan's."""
        key = ("accept", _sig(table), _sig(lengths), _sig(path), _sig(accepted), _sig(out))
        entry = self._seen.get(key)
        if entry is None:
            c, B = self.cache, self.B
            d = self._make_dims(*self._table(table), 0)
            c.check_ints(lengths, B, "lengths")
            c.check_ints(accepted, B, "accepted")
            if path.dtype != torch.int32 or path.device != self.device or tuple(path.shape) != (B, self.T) or \
                    not path.is_contiguous():
                raise ValueError(f"path: expected contiguous int32 ({B}, {self.T}) on {self.device}")
            if out is not None:
                c.check_ints(out, B, "out")
            if len(self._seen) >= 64:
                self._seen.clear()
            entry = self._seen[key] = (d, ctypes.byref(d))
        c = self.cache
        self._call(self._lib.paged_kv_accept, entry[1], c._kp, c._vp, table.data_ptr(), lengths.data_ptr(),
                   path.data_ptr(), accepted.data_ptr(), self._lengths_ptr if out is None else out.data_ptr(),
                   c._status_ptr)
        return self.lengths if out is None else out

    def read_status(self) -> int:
        """Synchronise and return the first failure that the plan's or the
        cache's device status word holds (0 = OK)."""
        own = capi.sca_read_status(self.status.data_ptr(), torch.cuda.current_stream(self.device).cuda_stream)
        return own or self.cache.read_status()
