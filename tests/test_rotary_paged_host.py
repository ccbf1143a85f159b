"""Rotary positions and the paged cache without a GPU: struct layouts, sizes of
workspaces, every refusal of the C entry points and of the constructors before
anything is launched (the addresses are never dereferenced), the frequencies
against their formulas, and the oracles against differences and plain
formulas."""
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
from sharded_causal_softmax_gb300.rotary import _TWO_PI, rotary_frequencies  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 30          # an aligned address that nothing reads
FAR = 1 << 40        # and one far behind it
BIG = 1 << 40        # bytes that are enough
V = capi.view
ARG, ALIGN, UNSUPPORTED = capi.SCA_ERR_ARG, capi.SCA_ERR_ALIGN, capi.SCA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from sharded_causal_softmax_gb300 import build
    build.build()
    return capi.lib()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_ctypes_structs_match_c_layout(tmp_path):
    structs = ("sca_rotary_dims", "sca_paged_dims")
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


# ------------------------------------------------------------------ rotary


def _rot(**kw):
    d = capi.sca_rotary_dims()
    d.B, d.H, d.Hkv, d.D, d.S, d.dtype, d.rotary_dim, d.amplitude = 2, 4, 2, 64, 10, capi.SCA_BF16, 32, 1.0
    d.q = d.qo = V(4 * 640, 640, 64)
    d.k = d.ko = V(2 * 640, 640, 64)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _apply(lib, d, q=A, k=A, turns=A, pos=None, qo=FAR, ko=FAR):
    return lib.rotary_apply(d and ctypes.byref(d), q, k, turns, pos, qo, ko, None)


@pytest.mark.parametrize("kw,code", [
    *[({f: x}, ARG) for f in ("B", "H") for x in (0, -1)], (dict(Hkv=-1), ARG), (dict(H=65535), ARG),
    *[(dict(S=x), ARG) for x in (0, -1, 1 << 31)], (dict(B=1 << 30, S=1 << 30), ARG),
    *[(dict(D=x), ARG) for x in (0, 63, 1026)], *[(dict(rotary_dim=x), ARG) for x in (-2, 3, 66)],
    (dict(dtype=3), ARG), (dict(amplitude=math.inf), ARG), (dict(amplitude=math.nan), ARG), (dict(pos_b=-1), ARG),
    (dict(q=V(-1, 640, 64)), ARG), (dict(k=V(1280, 640, 1 << 40)), ARG),
    # rows of an output over one another
    (dict(qo=V(2560, 640, 60)), ARG), (dict(qo=V(2560, 576, 64)), ARG), (dict(ko=V(640, 640, 64)), ARG),
    (dict(qo=V(0, 640, 64)), ARG), (dict(ko=V(64, 64, 64)), ARG),
])
def test_rotary_sizes_are_refused(lib, kw, code):
    assert _apply(lib, _rot(**kw)) == code
    assert b"rotary_apply" in lib.sca_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(d=None), ARG), *[({x: None}, ARG) for x in ("q", "k", "turns", "qo", "ko")],
    *[({x: A + 1}, ALIGN) for x in ("q", "k")], *[({x: FAR + 1}, ALIGN) for x in ("qo", "ko")],
    (dict(turns=A + 4), ALIGN), (dict(pos=A + 2), ALIGN),
    # an output over its input that is not the input itself
    (dict(qo=A + 2), ARG), (dict(qo=A + 2 * 2560), ARG), (dict(ko=A - 128), ARG),
    (dict(d=_rot(q=V(2560, 64, 256)), qo=A), ARG), (dict(d=_rot(q=V(0, 0, 0)), qo=A), ARG),
])
def test_rotary_calls_are_refused(lib, kw, code):
    kw = dict(kw)
    d = kw.pop("d", _rot())
    assert _apply(lib, d, **kw) == code


def test_two_pi_and_the_fixed_point_frequencies():
    # Machin's formula in integers of 200 bits
    one = 1 << 200

    def arctan(x):
        total, term, n = 0, one // x, 0
        while term:
            total += (term if n % 2 == 0 else -term) // (2 * n + 1)
            term //= x * x
            n += 1
        return total

    two_pi = 2 * 4 * (4 * arctan(5) - arctan(239))
    assert abs(int(_TWO_PI * one) - two_pi) < 1 << 73


@pytest.mark.parametrize("rd", [2, 4, 64, 128])
def test_frequencies(rd):
    f, a = rotary_frequencies(rd, base=500.0)
    i = np.arange(rd // 2)
    plain = np.exp(-np.log(500.0) * 2 * i / rd)
    np.testing.assert_allclose(f, plain, rtol=1e-14)
    assert a == 1.0
    np.testing.assert_allclose(rotary_frequencies(rd, 500.0, ("linear", 3.0))[0], plain / 3, rtol=1e-14)
    g, a = rotary_frequencies(rd, 500.0, ("base", 3.0))
    if rd > 2:   # the highest stays, the lowest is divided by the factor
        np.testing.assert_allclose([g[0], g[-1]], [plain[0], plain[-1] / 3], rtol=1e-12)
    g, a = rotary_frequencies(rd, 500.0, ("ramp", 8.0, 1000))
    turns = 1000 * plain / (2 * math.pi)
    assert a == pytest.approx(1 + 0.1 * math.log(8))
    for x, p, t in zip(g, plain, turns):
        part = min(max((t - 1) / 31, 0), 1)
        assert x == pytest.approx(p * part + p / 8 * (1 - part), rel=1e-13)
    for bad in (("linear",), ("linear", 0.5), ("linear", 2.0, 3), ("ramp", 2.0), ("ramp", 2.0, 0), ("ramp", 2.0, 9, 1),
                ("ramp", 2.0, 9, 5, 5), ("other", 2.0), ("base", math.nan)):
        with pytest.raises(ValueError):
            rotary_frequencies(rd, 500.0, bad)


def test_rotary_constructors_refuse():
    import sharded_causal_softmax_gb300 as sca
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(layout="other"), dict(base=0.0), dict(base=math.inf),
                dict(amplitude=math.nan), dict(frequencies=[1.0]), dict(frequencies=[1.0, math.inf]),
                dict(frequencies=[1.0, 2.0], scaling=("linear", 2.0)), dict(device="cpu")):
        with pytest.raises(ValueError):
            sca.RotaryAngles(**{**dict(rotary_dim=4, device="cuda:0"), **bad})


class Angles:   # what the constructors look at
    rotary_dim, device, layout, amplitude = 64, torch.device("cuda:0"), "half", 1.0


def test_plan_constructors_refuse():
    import sharded_causal_softmax_gb300 as sca
    ok = dict(B=2, H=4, S=10, D=64, angles=Angles())
    for bad in (dict(dtype=torch.float16), dict(B=0), dict(H=0), dict(kv_heads=0), dict(H=40000, kv_heads=30000),
                dict(S=0), dict(S=1 << 31), dict(D=63), dict(D=32), dict(D=1026), dict(device="cpu"),
                dict(device="cuda:1")):
        with pytest.raises(ValueError):
            sca.RotaryPositions(**{**ok, **bad})
    ok = dict(pages=4, kv_heads=2, D=64, device="cuda:0")
    for bad in (dict(dtype=torch.float16), dict(page=8), dict(page=48), dict(page=2048), dict(pages=0),
                dict(pages=1 << 31), dict(kv_heads=0), dict(D=60), dict(D=0), dict(D=1032), dict(device="cpu"),
                dict(D=32, angles=Angles()), dict(device="cuda:1", angles=Angles())):
        with pytest.raises(ValueError):
            sca.PagedKVCache(**{**ok, **bad})

    class Cache:
        Hkv, D, device, pages, page, dtype = 2, 64, torch.device("cuda:0"), 4, 16, torch.float32

    ok = dict(cache=Cache(), B=2, H=4)
    for bad in (dict(B=0), dict(H=0), dict(H=3), dict(B=40000), dict(tokens=0), dict(tokens=40000), dict(keys=0),
                dict(algo=capi.SCA_ALGO_TC)):
        with pytest.raises(ValueError):
            sca.PagedTreeAttention(**{**ok, **bad})


def test_rotary_oracle_turns_by_the_angle_and_its_transpose_undoes_it():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 5, 12))
    pos = rng.integers(-1000, 1000, (2, 5))
    f = rng.uniform(0, 3, 4)
    cos, sin = oracle.rotary_cos_sin(pos, f)
    np.testing.assert_allclose(cos, np.cos(pos[..., None] * f), atol=1e-11)
    np.testing.assert_allclose(sin, np.sin(pos[..., None] * f), atol=1e-11)
    cos, sin = cos[:, None], sin[:, None]
    for layout, (a, b) in (("half", (1, 5)), ("interleaved", (2, 3))):   # pair 1
        y = oracle.rotary(x, cos, sin, layout, 1.5)
        z = (x[..., a] + 1j * x[..., b]) * 1.5 * np.exp(1j * pos * f[1])[:, None]
        np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, atol=1e-11)
        assert np.array_equal(y[..., 8:], x[..., 8:])
        back = oracle.rotary(y, cos, sin, layout, 1.5, transposed=True)
        np.testing.assert_allclose(back[..., :8], 1.5 ** 2 * x[..., :8], atol=1e-12)


# ------------------------------------------------------------------- paged


def _dims(**kw):
    d = capi.sca_paged_dims()
    d.B, d.H, d.Hkv, d.T, d.D, d.dtype, d.algo, d.scale = 2, 8, 2, 4, 64, capi.SCA_BF16, capi.SCA_ALGO_AUTO, 0.125
    d.page, d.table_n, d.table_b, d.pages, d.pool = 16, 4000, 4000, 20, V(2 * 16 * 64, 16 * 64, 64)
    d.q, d.k, d.v = V(8 * 4 * 64, 4 * 64, 64), V(2 * 4 * 64, 4 * 64, 64), V(2 * 4 * 64, 4 * 64, 64)
    d.rotary_dim, d.amplitude, d.tree_b = 32, 1.0, 4
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _attend(lib, d, q=A, kp=A, vp=A, table=A, lengths=A, counts=None, tree=None, o=A, lse=A, ws=A, n=BIG):
    return lib.paged_tree_attend(d and ctypes.byref(d), q, kp, vp, table, lengths, counts, tree, o, lse, ws, n, None, None)


def _append(lib, d, q=A, k=A, v=A, table=A, lengths=A, counts=None, positions=None, turns=A, kp=FAR, vp=FAR, qo=FAR):
    return lib.paged_kv_append(d and ctypes.byref(d), q, k, v, table, lengths, counts, positions, turns, kp, vp, qo, None,
                               None)


def _accept(lib, d, kp=A, vp=A, table=A, lengths=A, path=A, accepted=A, out=A):
    return lib.paged_kv_accept(d and ctypes.byref(d), kp, vp, table, lengths, path, accepted, out, None, None)


CACHE = [
    *[({f: x}, ARG) for f in ("B", "Hkv", "T") for x in (0, -1)], (dict(B=40000), ARG), (dict(T=1 << 24), ARG),
    (dict(dtype=5), ARG), *[(dict(page=x), ARG) for x in (0, 8, 24, 48, 2048, -16)],
    *[(dict(pages=x), ARG) for x in (0, -1, 1 << 31)], (dict(table_n=0), ARG), (dict(table_n=1 << 27), ARG),
    (dict(table_b=-1), ARG), (dict(pool=V(2048, 1024, 56)), ARG), (dict(pool=V(-2048, 1024, 64)), ARG),
    (dict(pool=V(2048, 1 << 40, 64)), ARG), (dict(pool=V(2048, 1028, 64)), ALIGN), (dict(pool=V(2052, 1024, 64)), ALIGN),
    (dict(pool=V(2048, 1024, 68)), ALIGN),
]


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_sizes_are_refused(lib, kw, code):
    d, n = _dims(**kw), ctypes.c_int64()
    assert _attend(lib, d) == code and _append(lib, d) == code and _accept(lib, d) == code
    assert b"paged_kv_accept" in lib.sca_last_error()
    assert lib.paged_tree_workspace(ctypes.byref(d), ctypes.byref(n)) == code


@pytest.mark.parametrize("algo", [capi.SCA_ALGO_TC, capi.SCA_ALGO_SIMT])
@pytest.mark.parametrize("call,kw,code", [
    (_attend, dict(d=None), ARG), (_append, dict(d=None), ARG), (_accept, dict(d=None), ARG),
    *[(_attend, {x: None}, ARG) for x in ("q", "kp", "vp", "table", "lengths", "o", "lse", "ws")],
    *[(_append, {x: None}, ARG) for x in ("q", "k", "v", "table", "lengths", "turns", "kp", "vp", "qo")],
    *[(_accept, {x: None}, ARG) for x in ("kp", "vp", "table", "lengths", "path", "accepted", "out")],
    *[(_attend, {x: A + 8}, ALIGN) for x in ("q", "kp", "vp", "o", "ws")], (_attend, dict(tree=A + 4), ALIGN),
    *[(_attend, {x: A + 2}, ALIGN) for x in ("table", "lengths", "counts", "lse")],
    *[(_append, {x: A + 1}, ALIGN) for x in ("q", "k", "v")], *[(_append, {x: FAR + 8}, ALIGN) for x in ("kp", "vp", "qo")],
    *[(_append, {x: A + 2}, ALIGN) for x in ("table", "lengths", "counts", "positions", "turns")],
    *[(_accept, {x: A + 8}, ALIGN) for x in ("kp", "vp")],
    *[(_accept, {x: A + 2}, ALIGN) for x in ("table", "lengths", "path", "accepted", "out")],
    (_attend, dict(n=0), ARG), (_attend, dict(n=1000), ARG),
    (_attend, dict(dims=dict(H=0)), ARG), (_attend, dict(dims=dict(H=7)), ARG), (_attend, dict(dims=dict(H=1 << 16)), ARG),
    (_attend, dict(dims=dict(D=80, pool=V(2560, 1280, 80))), UNSUPPORTED), (_attend, dict(dims=dict(T=20000)), UNSUPPORTED),
    (_attend, dict(dims=dict(T=65, q=V(8 * 65 * 64, 0, 0)), tree=A), UNSUPPORTED),
    (_attend, dict(dims=dict(scale=0.0)), ARG), (_attend, dict(dims=dict(scale=math.nan)), ARG),
    (_attend, dict(dims=dict(q=V(2040, 0, 0))), ARG), (_attend, dict(dims=dict(q=V(2052, 0, 0))), ALIGN),
    (_attend, dict(dims=dict(tree_b=-1)), ARG), (_attend, dict(dims=dict(algo=7)), ARG),
    (_attend, dict(dims=dict(dtype=capi.SCA_F32, algo=capi.SCA_ALGO_TC)), UNSUPPORTED),
    (_append, dict(dims=dict(rotary_dim=66)), ARG), (_append, dict(dims=dict(rotary_dim=3)), ARG),
    (_append, dict(dims=dict(amplitude=math.inf)), ARG), (_append, dict(dims=dict(pos_b=-1)), ARG),
    (_append, dict(dims=dict(H=40000)), ARG), (_append, dict(dims=dict(k=V(-1, 0, 0))), ARG),
    (_append, dict(dims=dict(v=V(1 << 40, 0, 0))), ARG),
    # pools whose rows share elements may be read, not written
    (_append, dict(dims=dict(pool=V(1024, 1024, 64))), ARG), (_accept, dict(dims=dict(pool=V(2048, 0, 64))), ARG),
    (_append, dict(dims=dict(pool=V(0, 1024, 64))), ARG),
])
def test_paged_calls_are_refused(lib, call, kw, code, algo):
    kw = dict(kw)
    d = kw.pop("d") if "d" in kw else _dims(**{**dict(algo=algo), **kw.pop("dims", {})})
    assert call(lib, d, **kw) == code


def test_workspace_of_a_plan_serves_shorter_tables(lib):
    for algo in (capi.SCA_ALGO_AUTO, capi.SCA_ALGO_SIMT, capi.SCA_ALGO_TC):
        for kw in (dict(), dict(T=64, q=V(8 * 64 * 64, 0, 0)), dict(B=300, H=2), dict(B=1, H=2, T=1)):
            most = capi.paged_tree_workspace(_dims(table_n=5000, algo=algo, **kw))
            assert all(capi.paged_tree_workspace(_dims(table_n=n, algo=algo, **kw)) <= most for n in (1, 2, 7, 100, 499, 4999))
    assert lib.paged_tree_workspace(ctypes.byref(_dims()), None) == ARG


@pytest.mark.parametrize("dtype", [capi.SCA_BF16, capi.SCA_F32])
@pytest.mark.parametrize("D", [64, 128])
def test_no_shorter_table_needs_a_larger_workspace(lib, dtype, D):
    ask = lambda n, B, Hkv, T: capi.paged_tree_workspace(_dims(
        table_n=n, B=B, H=Hkv, Hkv=Hkv, T=T, D=D, dtype=dtype, page=16, table_b=n, q=V(Hkv * T * D, 0, 0),
        pool=V(Hkv * 16 * D, 16 * D, D)))
    for B in (1, 2, 3, 19, 38, 76, 152):
        for Hkv in (1, 2, 8):
            for T in (1, 4, 8, 16, 17, 64):
                sizes = [ask(n, B, Hkv, T) for n in (1, 2, 3, 5, 9, 17, 33, 64, 100, 128, 200, 256, 400, 777, 1600, 6000)]
                assert all(max(sizes[:i]) <= sizes[i] for i in range(1, len(sizes))), (B, Hkv, T, sizes)


def test_paged_oracle_is_softmax_over_the_gathered_rows():
    g = torch.Generator().manual_seed(5)
    B, H, Hkv, T, D, page = 2, 4, 2, 3, 8, 4
    kp, vp = (torch.randn(9, Hkv, page, D, generator=g, dtype=torch.float64) for _ in range(2))
    table, lengths, counts = torch.tensor([[3, 0, 8], [5, 1, 2]]), [5, 0], [3, 2]
    tree = [[0b001, 0b011, 0b101], [0b01, 0b10, 0b0]]
    q = torch.randn(B, H, T, D, generator=g, dtype=torch.float64)
    o, lse, _ = oracle.tree_attention(q, kp, vp, table, lengths, counts, tree, 0.4)
    for b in range(B):
        k, v = (p[table[b]].transpose(0, 1).reshape(Hkv, -1, D).repeat_interleave(H // Hkv, 0) for p in (kp, vp))
        j = torch.arange(3 * page) - lengths[b]
        for t in range(counts[b]):
            seen = torch.tensor([x < 0 or (x < counts[b] and bool(tree[b][t] >> x & 1)) for x in j.tolist()])
            s = (0.4 * q[b, :, t, None] @ k.transpose(-1, -2))[:, 0].masked_fill(~seen, -math.inf)
            np.testing.assert_allclose(o[b, :, t], (s.softmax(-1)[:, None] @ v)[:, 0], rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(lse[b, :, t], s.logsumexp(-1), rtol=1e-12, atol=1e-13)
    assert not o[1, :, 2].any() and np.isneginf(lse[1, :, 2]).all()
    # rows appended one by one, and a path kept
    new = torch.randn(B, Hkv, T, D, generator=g, dtype=torch.float64).numpy()
    pool = oracle.paged_append(kp.numpy(), new, table, lengths, counts)
    assert np.array_equal(pool[8], kp[8].numpy()) and np.array_equal(pool[0][:, 1:4], new[0])
    assert np.array_equal(pool[5][:, :2], new[1][:, :2]) and np.array_equal(pool[5][:, 2:], kp[5][:, 2:].numpy())
    kept = oracle.paged_accept(pool, table, lengths, [[0, 2, 0], [1, 0, 0]], [2, 1])
    assert np.array_equal(kept[0][:, 1:3], new[0][:, [0, 2]]) and np.array_equal(kept[5][:, 0], new[1][:, 1])
