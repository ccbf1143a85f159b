"""Decaying linear attention and shared-prefix decoding without a GPU: struct
layouts, sizes of workspaces, every refusal of the C entry points and of the
plans' constructors before anything is launched (the addresses are never
dereferenced), and the oracles against differences and plain formulas."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle

capi = pytest.importorskip("sharded_causal_softmax_gb300.capi")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 30          # an aligned address that nothing reads
FAR = 1 << 40        # and one far behind it
BIG = 1 << 40        # bytes that are enough


@pytest.fixture(scope="module")
def lib():
    from sharded_causal_softmax_gb300 import build
    build.build()
    return capi.lib()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_ctypes_structs_match_c_layout(tmp_path):
    structs = ("sca_decay_dims", "sca_prefix_dims")
    lines = []
    for s in structs:
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for f, _ in getattr(capi, s)._fields_]
    src = tmp_path / "probe.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"sca.h\"\nint main(void) {\n" + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    seen = dict(line.rsplit(" ", 1) for line in out if line)
    assert len(seen) == len(lines)
    for key, val in seen.items():
        s, _, f = key.partition(".")
        mine = getattr(getattr(capi, s), f).offset if f else ctypes.sizeof(getattr(capi, s))
        assert mine == int(val), key


# ------------------------------------------------------------------- decay


def _decay(**kw):
    d = capi.sca_decay_dims()
    d.B, d.H, d.D, d.dtype, d.algo, d.scale, d.S = 2, 3, 64, capi.SCA_BF16, capi.SCA_ALGO_AUTO, 0.125, 300
    d.q = d.k = d.v = d.o = capi.view(3 * 300 * 64, 300 * 64, 64)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


ONE = 3 * 64 * 64    # floats of a sequence's states
V = capi.view
BAD_DIMS = [
    (dict(B=0), capi.SCA_ERR_ARG), (dict(H=0), capi.SCA_ERR_ARG), (dict(B=-1), capi.SCA_ERR_ARG),
    (dict(B=256, H=256), capi.SCA_ERR_ARG), (dict(D=96), capi.SCA_ERR_UNSUPPORTED), (dict(D=0), capi.SCA_ERR_UNSUPPORTED),
    (dict(dtype=7), capi.SCA_ERR_ARG), (dict(algo=9), capi.SCA_ERR_ARG), (dict(algo=-1), capi.SCA_ERR_ARG),
    (dict(dtype=capi.SCA_F32, algo=capi.SCA_ALGO_TC), capi.SCA_ERR_UNSUPPORTED),
    (dict(scale=math.inf), capi.SCA_ERR_ARG), (dict(scale=math.nan), capi.SCA_ERR_ARG),
    (dict(q=V(-8, 19200, 64)), capi.SCA_ERR_ARG), (dict(k=V(57600, -64, 64)), capi.SCA_ERR_ARG),
    (dict(v=V(57601, 19200, 64)), capi.SCA_ERR_ALIGN), (dict(q=V(57600, 19204, 64)), capi.SCA_ERR_ALIGN),
]
BAD_ROWS = [
    (dict(S=0), capi.SCA_ERR_ARG), (dict(S=-5), capi.SCA_ERR_ARG), (dict(S=1 << 24), capi.SCA_ERR_ARG),
    (dict(q=V(57600, 19200, 56)), capi.SCA_ERR_ARG), (dict(k=V(57600, 19200, 68)), capi.SCA_ERR_ALIGN),
    (dict(o=V(57600, 19200, 68)), capi.SCA_ERR_ALIGN), (dict(o=V(57600, 19200, 32)), capi.SCA_ERR_ARG),
]


def _fwd(lib, d, q=A, k=A, v=A, g=A, lengths=None, s=None, sb=0, o=A, end=FAR, ws=A, n=BIG):
    return lib.decay_attn_fwd(d and ctypes.byref(d), q, k, v, g, lengths, s, sb, o, end, ws, n, None, None)


def _bwd(lib, d, q=A, k=A, v=A, do=A, dov=V(57600, 19200, 64), g=A, s=None, sb=0, ds=None, db=0, dq=A, dk=A, dv=A,
         ds0=None, ws=A, n=BIG):
    return lib.decay_attn_bwd(d and ctypes.byref(d), q, k, v, do, dov and ctypes.byref(dov), g, None, s, sb, ds, db,
                              dq, dk, dv, ds0, ws, n, 0, None, None)


def _step(lib, d, q=A, k=A, v=A, g=A, s=A, sb=ONE, o=A):
    return lib.decay_attn_step(d and ctypes.byref(d), q, k, v, g, s, sb, o, None)


@pytest.mark.parametrize("kw,code", BAD_DIMS + BAD_ROWS)
def test_decay_sizes_are_refused(lib, kw, code):
    d, n = _decay(**kw), ctypes.c_int64()
    assert lib.decay_attn_workspace(ctypes.byref(d), 0, ctypes.byref(n)) == code
    assert _fwd(lib, d) == code and _bwd(lib, d) == code
    assert b"decay_attn_bwd" in lib.sca_last_error()
    if (kw, code) in BAD_DIMS:
        assert _step(lib, d) == code
    assert lib.decay_attn_workspace(None, 0, ctypes.byref(n)) == capi.SCA_ERR_ARG
    assert lib.decay_attn_workspace(ctypes.byref(_decay()), 0, None) == capi.SCA_ERR_ARG


def test_decay_fp32_strides_need_four_elements(lib):
    d = _decay(dtype=capi.SCA_F32, q=V(57600, 19200, 66))
    assert _fwd(lib, d) == capi.SCA_ERR_ALIGN


@pytest.mark.parametrize("call,kw,code", [
    (_fwd, dict(d=None), capi.SCA_ERR_ARG), (_bwd, dict(d=None), capi.SCA_ERR_ARG), (_step, dict(d=None), capi.SCA_ERR_ARG),
    *[(_fwd, {x: None}, capi.SCA_ERR_ARG) for x in ("q", "k", "v", "g", "o", "end")],
    *[(_bwd, {x: None}, capi.SCA_ERR_ARG) for x in ("q", "k", "v", "do", "dov", "g", "dq", "dk", "dv")],
    *[(_step, {x: None}, capi.SCA_ERR_ARG) for x in ("q", "k", "v", "g", "s", "o")],
    *[(_fwd, {x: A + 8}, capi.SCA_ERR_ALIGN) for x in ("q", "k", "v", "o", "end", "s", "ws")],
    *[(_bwd, {x: A + 8}, capi.SCA_ERR_ALIGN) for x in ("q", "k", "v", "do", "dq", "dk", "dv", "s", "ds", "ds0", "ws")],
    *[(_step, {x: A + 8}, capi.SCA_ERR_ALIGN) for x in ("q", "k", "v", "s", "o")],
    (_fwd, dict(s=A, sb=ONE - 4), capi.SCA_ERR_ARG), (_fwd, dict(s=A, sb=-ONE), capi.SCA_ERR_ARG),
    (_fwd, dict(s=A, sb=ONE + 1), capi.SCA_ERR_ALIGN),
    # the end state over the first: only as the same states
    (_fwd, dict(s=FAR, sb=0), capi.SCA_ERR_ARG), (_fwd, dict(s=FAR, sb=ONE + 4), capi.SCA_ERR_ARG),
    (_fwd, dict(s=FAR + 64, sb=ONE), capi.SCA_ERR_ARG), (_fwd, dict(s=FAR - 8 * ONE + 16, sb=ONE), capi.SCA_ERR_ARG),
    (_bwd, dict(ds=A, db=ONE - 4), capi.SCA_ERR_ARG), (_bwd, dict(dov=V(57600, 19200, 60)), capi.SCA_ERR_ARG),
    (_bwd, dict(dov=V(57600, 19200, 68)), capi.SCA_ERR_ALIGN), (_bwd, dict(dov=V(-64, 19200, 64)), capi.SCA_ERR_ARG),
    (_bwd, dict(ds=FAR, db=ONE, ds0=FAR), capi.SCA_ERR_ARG), (_bwd, dict(ds=FAR, db=0, ds0=FAR + 64), capi.SCA_ERR_ARG),
    (_bwd, dict(s=FAR, sb=ONE, ds0=FAR), capi.SCA_ERR_ARG), (_bwd, dict(s=FAR, sb=0, ds0=FAR), capi.SCA_ERR_ARG),
    (_step, dict(sb=0), capi.SCA_ERR_ARG), (_step, dict(sb=ONE - 4), capi.SCA_ERR_ARG),
    (_step, dict(sb=ONE + 2), capi.SCA_ERR_ALIGN),
])
def test_decay_calls_are_refused(lib, call, kw, code):
    kw = dict(kw)
    d = kw.pop("d", _decay())
    assert call(lib, d, **kw) == code


@pytest.mark.parametrize("dtype", [capi.SCA_BF16, capi.SCA_F32])
def test_decay_workspace_is_asked_for_and_checked(lib, dtype):
    need = []
    for S in (1, 128, 129, 5000, 100000):
        d = _decay(S=S, dtype=dtype, q=V(3 * S * 64, S * 64, 64), B=1, H=3)
        one, two = capi.decay_attn_workspace(d, 0), capi.decay_attn_workspace(d, 1)
        assert two == 2 * one and one % (3 * 64 * 64 * 4) == 0
        need.append(one)
        if S == 100000:
            for n in (0, 1024):
                assert _fwd(lib, d, n=n) == capi.SCA_ERR_ARG and _bwd(lib, d, n=n) == capi.SCA_ERR_ARG
            assert _fwd(lib, d, ws=None) == capi.SCA_ERR_ARG and _bwd(lib, d, ws=None) == capi.SCA_ERR_ARG
    # fewer rows never need more; what segments hold grows with a fill of the SMs, not with S
    assert need == sorted(need) and need[-1] <= 3 * 64 * 64 * 4 * 320


def test_decay_plan_refusals():
    import sharded_causal_softmax_gb300 as sca
    ok = dict(B=2, H=3, S=64, D=64, log_decay=[-0.1, -0.2, 0.0], device="cuda:0")
    for bad in (dict(dtype=torch.float16), dict(D=96), dict(B=0), dict(B=40000), dict(S=0), dict(S=1 << 24),
                dict(dtype=torch.float32, algo=capi.SCA_ALGO_TC), dict(device="cpu"), dict(log_decay=[-0.1, -0.2]),
                dict(log_decay=[-0.1, 0.1, 0.0]), dict(log_decay=[-0.1, math.nan, 0.0]), dict(scale=math.nan)):
        with pytest.raises(ValueError):
            sca.DecayLinearAttention(**{**ok, **bad})


def test_decay_oracle_is_the_sum_over_earlier_rows_and_its_gradient():
    rng = np.random.default_rng(3)
    B, H, S, D, scale, lengths = 2, 2, 7, 4, 0.3, [7, 4]
    q, k, v, do = (rng.standard_normal((B, H, S, D)) for _ in range(4))
    s0, ds = (rng.standard_normal((B, H, D, D)) for _ in range(2))
    g = np.array([-0.2, -1.1])
    o, end = oracle.decay_attention(q, k, v, g, scale, s0, lengths)
    for b in range(B):
        for h in range(H):
            for t in range(S):
                want = np.zeros(D)
                if t < lengths[b]:
                    want = math.exp(g[h] * (t + 1)) * q[b, h, t] @ s0[b, h]
                    for s in range(t + 1):
                        want = want + math.exp(g[h] * (t - s)) * (q[b, h, t] @ k[b, h, s]) * v[b, h, s]
                np.testing.assert_allclose(o[b, h, t], scale * want, rtol=1e-12, atol=1e-13)

    def loss(q, k, v, s0):
        o, end = oracle.decay_attention(q, k, v, g, scale, s0, lengths)
        return (o * do).sum() + (end * ds).sum()

    grads = oracle.decay_attention_backward(q, k, v, do, g, scale, s0, ds, lengths)
    xs = [q, k, v, s0]
    h = 1e-5   # the loss is a polynomial of degree 3 with terms of order one: h^2 and rounding / h are below 1e-8
    for i, grad in enumerate(grads):
        for at in [tuple(rng.integers(n) for n in xs[i].shape) for _ in range(40)]:
            up, down = [x.copy() for x in xs], [x.copy() for x in xs]
            up[i][at] += h
            down[i][at] -= h
            assert abs((loss(*up) - loss(*down)) / (2 * h) - grad[at]) < 1e-7 * (1 + abs(grad[at]))


# ------------------------------------------------------------------ prefix


def _prefix(**kw):
    d = capi.sca_prefix_dims()
    d.B, d.H, d.Hkv, d.T, d.D, d.dtype, d.algo, d.scale = 2, 8, 2, 2, 64, capi.SCA_BF16, capi.SCA_ALGO_AUTO, 0.125
    d.q_b, d.prefix_len, d.suffix_cap = 8 * 2 * 64, 500, 200
    d.prefix, d.suffix = V(0, 500 * 64, 64), V(2 * 200 * 64, 200 * 64, 64)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _decode(lib, d, q=A, kp=A, vp=A, ks=A, vs=A, lengths=A, o=A, lse=A, ws=A, n=BIG):
    return lib.prefix_attn_decode(d and ctypes.byref(d), q, kp, vp, ks, vs, lengths, o, lse, ws, n, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), capi.SCA_ERR_ARG), (dict(H=0), capi.SCA_ERR_ARG), (dict(Hkv=0), capi.SCA_ERR_ARG),
    (dict(Hkv=3), capi.SCA_ERR_ARG), (dict(T=0), capi.SCA_ERR_ARG), (dict(B=16384), capi.SCA_ERR_ARG),
    (dict(T=33, q_b=8 * 33 * 64), capi.SCA_ERR_UNSUPPORTED), (dict(H=258, q_b=258 * 128), capi.SCA_ERR_UNSUPPORTED),
    (dict(D=80), capi.SCA_ERR_UNSUPPORTED), (dict(dtype=5), capi.SCA_ERR_ARG), (dict(algo=3), capi.SCA_ERR_ARG),
    (dict(dtype=capi.SCA_F32, algo=capi.SCA_ALGO_TC), capi.SCA_ERR_UNSUPPORTED),
    (dict(scale=0.0), capi.SCA_ERR_ARG), (dict(scale=-0.1), capi.SCA_ERR_ARG), (dict(scale=math.nan), capi.SCA_ERR_ARG),
    (dict(scale=math.inf), capi.SCA_ERR_ARG), (dict(prefix_len=-1), capi.SCA_ERR_ARG),
    (dict(prefix_len=1 << 31), capi.SCA_ERR_ARG), (dict(suffix_cap=-1), capi.SCA_ERR_ARG),
    (dict(suffix_cap=(1 << 31) - 128), capi.SCA_ERR_ARG), (dict(q_b=8 * 2 * 64 - 8), capi.SCA_ERR_ARG),
    (dict(q_b=-1024), capi.SCA_ERR_ARG), (dict(q_b=8 * 2 * 64 + 4), capi.SCA_ERR_ALIGN),
    (dict(prefix=V(0, 500 * 64, 56)), capi.SCA_ERR_ARG), (dict(prefix=V(0, 500 * 64, 68)), capi.SCA_ERR_ALIGN),
    (dict(prefix=V(0, -64, 64)), capi.SCA_ERR_ARG), (dict(suffix=V(0, 0, 63)), capi.SCA_ERR_ARG),
    (dict(suffix=V(25604, 12800, 64)), capi.SCA_ERR_ALIGN),
])
def test_prefix_sizes_are_refused(lib, kw, code):
    d, n = _prefix(**kw), ctypes.c_int64()
    assert lib.prefix_attn_workspace(ctypes.byref(d), ctypes.byref(n)) == code
    assert _decode(lib, d) == code
    assert b"prefix_attn" in lib.sca_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(d=None), capi.SCA_ERR_ARG),
    *[({x: None}, capi.SCA_ERR_ARG) for x in ("q", "kp", "vp", "ks", "vs", "lengths", "o", "lse", "ws")],
    *[({x: A + 8}, capi.SCA_ERR_ALIGN) for x in ("q", "kp", "vp", "ks", "vs", "o", "ws")],
    *[({x: A + 2}, capi.SCA_ERR_ALIGN) for x in ("lse", "lengths")],
    (dict(n=0), capi.SCA_ERR_ARG), (dict(n=1000), capi.SCA_ERR_ARG),
])
@pytest.mark.parametrize("algo", [capi.SCA_ALGO_AUTO, capi.SCA_ALGO_SIMT])
def test_prefix_calls_are_refused(lib, kw, code, algo):
    kw = dict(kw)
    d = kw.pop("d", _prefix(algo=algo))
    assert _decode(lib, d, **kw) == code


def test_prefix_line_of_tiles_has_a_limit(lib):
    # 4095 requests x 16 heads x 2^24 tiles of a suffix: places on the line pass 32 bits
    d = _prefix(B=4095, H=16, Hkv=16, T=1, q_b=16 * 64, suffix_cap=(1 << 31) - 200, suffix=V(0, 0, 64))
    assert _decode(lib, d, n=1 << 62) == capi.SCA_ERR_UNSUPPORTED


@pytest.mark.parametrize("algo", [capi.SCA_ALGO_AUTO, capi.SCA_ALGO_SIMT])
def test_prefix_workspace_of_a_plan_serves_shorter_caches(lib, algo):
    most = capi.prefix_attn_workspace(_prefix(prefix_len=5000, suffix_cap=700, algo=algo))
    for p in (0, 1, 127, 128, 129, 1000, 3333, 4999, 5000):
        for s in (0, 1, 128, 129, 500, 700):
            assert capi.prefix_attn_workspace(_prefix(prefix_len=p, suffix_cap=s, algo=algo)) <= most


def test_prefix_plan_refusals():
    import sharded_causal_softmax_gb300 as sca
    ok = dict(B=2, H=8, D=64, prefix=100, suffix=50, kv_heads=2, tokens=2, device="cuda:0")
    for bad in (dict(dtype=torch.float16), dict(D=32), dict(kv_heads=3), dict(B=0), dict(B=20000), dict(tokens=0),
                dict(tokens=33), dict(prefix=-1), dict(suffix=-1), dict(dtype=torch.float32, algo=capi.SCA_ALGO_TC),
                dict(device="cpu"), dict(scale=0.0), dict(scale=math.inf)):
        with pytest.raises(ValueError):
            sca.SharedPrefixAttention(**{**ok, **bad})


def test_prefix_oracle_is_softmax_over_both_caches():
    g = torch.Generator().manual_seed(5)
    B, H, Hkv, T, D, n, cap, lengths = 2, 4, 2, 3, 8, 5, 6, [6, 2]
    q = torch.randn(B, H, T, D, generator=g, dtype=torch.float64)
    kp, vp = (torch.randn(Hkv, n, D, generator=g, dtype=torch.float64) for _ in range(2))
    ks, vs = (torch.randn(B, Hkv, cap, D, generator=g, dtype=torch.float64) for _ in range(2))
    o, lse, _ = oracle.prefix_decode(q, kp, vp, ks, vs, lengths, 0.4)
    for b in range(B):
        k = torch.cat((kp, ks[b]), 1).repeat_interleave(H // Hkv, 0)
        v = torch.cat((vp, vs[b]), 1).repeat_interleave(H // Hkv, 0)
        j = torch.arange(n + cap)
        seen = (j[None] < n) | (j[None] - n < lengths[b] - (T - 1 - torch.arange(T))[:, None])
        s = (0.4 * q[b] @ k.transpose(-1, -2)).masked_fill(~seen, -math.inf)
        np.testing.assert_allclose(o[b], s.softmax(-1) @ v, rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(lse[b], s.logsumexp(-1), rtol=1e-12, atol=1e-13)
