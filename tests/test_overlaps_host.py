"""Tensors that share bytes, without a GPU: the test for it against the bytes
themselves, and the calls of the rotary and paged entry points that it refuses
(the addresses are never dereferenced)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

capi = pytest.importorskip("sharded_causal_softmax_gb300.capi")
from tests.test_rotary_paged_host import ARG, FAR, V, _accept, _append, _apply, _dims, _rot, lib  # noqa: E402,F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 30
CODE = r"""
#include <cstdio>
#include "disjoint.h"
int main() {
  sca::Rows r[2];
  long long base, n[3], s[3], bytes;
  while (true) {
    for (int i = 0; i < 2; ++i) {
      if (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &base, &bytes, s, s + 1, s + 2, n, n + 1, n + 2) != 8) return 0;
      r[i] = {reinterpret_cast<const void*>(base), bytes, {s[0], s[1], s[2]}, {n[0], n[1], n[2]}};
    }
    std::printf("%d %d\n", sca::share_bytes(r[0], r[1]), sca::share_bytes(r[1], r[0]));
  }
}
"""


def answers(tmp_path, pairs):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(CODE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "sharded_causal_softmax_gb300", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    text = "\n".join(" ".join(str(x) for x in (base, bytes_, *s, *n)) for pair in pairs for base, bytes_, s, n in pair)
    out = subprocess.run([str(exe)], input=text + "\n", capture_output=True, text=True, check=True).stdout.split("\n")
    got = [tuple(int(x) for x in line.split()) for line in out if line]
    assert len(got) == len(pairs) and all(a == b for a, b in got)
    return [bool(a) for a, _ in got]


def bytes_of(base, size, s, n):
    return {base + i * s[0] + j * s[1] + k * s[2] + e for i in range(n[0]) for j in range(n[1]) for k in range(n[2])
            for e in range(size)}


def test_shared_bytes_are_those_that_both_hold(tmp_path):
    rng = random.Random(3)
    pairs = []
    for _ in range(3000):
        strides = [rng.choice((0, 1, 2, 3, 4, 6, 8, 12, 16, 20, 24, 48, 60, 120)) for _ in range(6)]
        if rng.random() < 0.5:
            strides[3:] = strides[:3]       # views of one tensor
        pairs.append(tuple((1000 + rng.randrange(80 if i else 8), rng.choice((1, 2, 4, 7)), strides[3 * i:3 * i + 3],
                            [rng.randint(1, 6) for _ in range(3)]) for i in range(2)))
    want = [bool(bytes_of(*a) & bytes_of(*b)) for a, b in pairs]
    assert 500 < sum(want) < 2500
    assert answers(tmp_path, pairs) == want


def test_views_of_real_sizes(tmp_path):
    """Queries and keys of one projection, pools of keys and values between one
    another, a layer of a pool of many: apart, until one is moved by a row."""
    B, S, H, Hkv, D = 64, 32768, 32, 8, 256            # bytes of a row
    W = (H + 2 * Hkv) * D
    q = (A, D, (S * W, D, W), (B, H, S))
    k = (A + H * D, D, (S * W, D, W), (B, Hkv, S))
    pages, page, layers = 1 << 20, 64, 80
    kv = [(A + i * Hkv * page * D, D, (2 * Hkv * page * D, page * D, D), (pages, Hkv, page)) for i in range(2)]
    rows = [(A + i * Hkv * D, D, (page * 2 * Hkv * D, D, 2 * Hkv * D), (pages, Hkv, page)) for i in range(2)]
    layer = [(A + (2 * x + i) * Hkv * page * D, D, (2 * layers * Hkv * page * D, page * D, D), (pages, Hkv, page))
             for x, i in ((0, 0), (0, 1), (79, 1))]
    by = lambda t, n: (t[0] + n, *t[1:])
    gap = (layer[1][0] + 2 * Hkv * page * D + 64, D, (8 * 4 * D, 4 * D, D), (B, 8, 4))   # inside the next layer
    end = (FAR, D, (1 << 42, 1 << 42, 1 << 42), (1 << 30, 65535, 1 << 30))              # past 64 bits
    pairs = [(q, k), (q, by(k, -1)), (q, by(k, -D)), kv, (kv[0], by(kv[1], -16)), rows, (rows[0], by(rows[1], -D)),
             layer[:2], (layer[1], layer[2]), (layer[0], gap), (layer[1], gap), (end, by(end, D)), (end, by(end, D - 1))]
    assert answers(tmp_path, pairs) == [False, True, True, False, True, False, True, False, False, False, False, False, True]


def test_rotary_outputs_over_the_other_tensor_are_refused(lib):
    assert _apply(lib, _rot(), q=A, k=FAR, qo=A, ko=A + 2 * 640) == ARG            # over one another
    assert _apply(lib, _rot(), q=A, k=FAR, qo=FAR, ko=2 * FAR) == ARG              # qo over k
    assert _apply(lib, _rot(), q=A, k=FAR, qo=2 * FAR, ko=A + 2 * 4 * 640) == ARG  # ko over q
    assert b"overlaps the other" in lib.sca_last_error()
    # out of one projection [B, S, H + Hkv, D], the view of the output off by a head
    view = V(10 * 6 * 64, 64, 6 * 64)
    d = _rot(q=view, qo=view, k=view, ko=view)
    assert _apply(lib, d, q=A, k=A + 2 * 4 * 64, qo=A, ko=A + 2 * 3 * 64) == ARG


def test_appends_over_their_own_inputs_are_refused(lib):
    T = 4
    apart = dict(q=A, k=2 * FAR, v=3 * FAR, kp=4 * FAR, vp=5 * FAR, qo=6 * FAR)
    for at, over in (("qo", "q"), ("qo", "k"), ("qo", "v"), ("qo", "kp"), ("qo", "vp"), ("kp", "k"), ("kp", "v"),
                     ("kp", "q"), ("vp", "k"), ("vp", "v"), ("vp", "q"), ("vp", "kp")):
        assert _append(lib, _dims(), **{**apart, at: apart[over] + 128}) == ARG, (at, over)
        assert b"overlap" in lib.sca_last_error()
    # queries in place only where they lie as the output does
    for view in (V(8 * T * 64, 64, 8 * 64), V(0, T * 64, 64), V(8 * T * 64, T * 64, 128)):
        assert _append(lib, _dims(q=view), **{**apart, "qo": A}) == ARG
    assert _accept(lib, _dims(), kp=A, vp=A) == ARG
    assert _accept(lib, _dims(), kp=A, vp=A + 16 * 64) == ARG
