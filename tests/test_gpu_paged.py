"""GPU parity of the paged cache (append, attention of drafted tokens,
acceptance) against the fp64 oracle.

Bounds of the attention: o = sum_j p_j v_j / sum_j p_j with A = sum_j p_j |v_j|
/ sum_j p_j.  The tensor-core kernel rounds each p_j to bf16 for the product
with V (half a step, 2^-8 of A at most); scores are fp32 sums of exact products,
off by at most es = D 2^-23 |q| |k| scale (2-norms), which moves a weight by as
much, each way; fp32 sums over n rows add n 2^-23 of A (the tensor cores
truncate); the output adds half a step of its type.  lse is a log: its absolute
error is the relative one of the sum, plus half a step of itself.  Appended keys
are held to the rotation's bound (tests/test_gpu_rotary.py), values and accepted
rows to their bits."""
import math
import random

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sca():
    import sharded_causal_softmax_gb300 as m
    from sharded_causal_softmax_gb300 import build
    build.build()
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def make_tree(B, T, seed, reach=5):
    """(words, parents) of random trees."""
    rng = random.Random(seed)
    words, parents = [], []
    for _ in range(B):
        w, ps = [], []
        for t in range(T):
            p = rng.randint(max(-1, t - reach), t - 1) if t else -1
            ps.append(p)
            w.append((w[p] if p >= 0 else 0) | 1 << t)
        words.append([x - (1 << 64) if x >> 63 else x for x in w])
        parents.append(ps)
    return torch.tensor(words, dtype=torch.int64), parents


class Setup:
    """A pool in use, tables that scatter each request's pages over it, and NaN
    in every row that no request holds."""

    def __init__(self, B, Hkv, group, T, D, page, lengths, counts, dtype, seed, spare=2, extra=3):
        g = torch.Generator().manual_seed(seed)
        self.rnd = lambda *s: torch.randn(*s, generator=g).to(dtype)
        self.B, self.Hkv, self.H, self.T, self.D, self.page, self.dtype = B, Hkv, Hkv * group, T, D, page, dtype
        self.lengths, self.counts = lengths, [T] * B if counts is None else counts
        each = -(-(max(max(lengths), 0) + T) // page) + spare
        self.pages = B * each + extra
        self.table = torch.randperm(self.pages, generator=g)[:B * each].to(torch.int32).reshape(B, each)
        self.k, self.v = self.rnd(self.pages, Hkv, page, D), self.rnd(self.pages, Hkv, page, D)
        used = torch.zeros(self.pages, page, dtype=torch.bool)
        for b in range(B):
            at = torch.arange(max(0, lengths[b]) + max(0, min(T, self.counts[b])))
            used[self.table[b].long()[at // page], at % page] = True
        self.k.transpose(1, 2)[~used] = float("nan")
        self.v.transpose(1, 2)[~used] = float("inf")
        # entries behind the pages that a request needs may be anything
        for b in range(B):
            need = -(-(max(0, lengths[b]) + max(0, min(T, self.counts[b]))) // page)
            self.table[b, need:] = torch.tensor([-7, 1 << 30] * each, dtype=torch.int32)[:each - need]
        self.q = self.rnd(B, self.H, T, D)

    def cache(self, sca, **kw):
        return sca.PagedKVCache(self.pages, self.Hkv, self.D, page=self.page, dtype=self.dtype,
                                pools=(self.k.cuda(), self.v.cuda()), **kw)


def compare(o, lse, s, tree, scale, tc, q=None):
    q = s.q if q is None else q
    words = None if tree is None else [[int(x) for x in row] for row in tree.expand(s.B, s.T).tolist()]
    ref, rl, mag = oracle.tree_attention(q, s.k, s.v, s.table, s.lengths, s.counts, words, scale)
    n = max(max(0, x) for x in s.lengths) + s.T
    kmax = float(torch.nan_to_num(s.k.double(), nan=0.0).norm(dim=-1).max())
    es = s.D * 2.0 ** -23 * float(q.double().norm(dim=-1).max()) * kmax * scale + 2.0 ** -21
    err = 2 * es + n * 2.0 ** -23 + 2.0 ** -20 + (2.0 ** -8 if tc else 0.0)
    g, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl)) and np.isfinite(g).all()
    bound = HALF[s.dtype] * 1.01 * np.abs(ref) + err * mag
    assert (np.abs(g - ref) <= bound).all(), f"o: {(np.abs(g - ref) / np.maximum(bound, 1e-37)).max():.2f} of the bound"
    seen = ~np.isneginf(rl)
    lb = es + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * np.abs(rl[seen])
    assert (np.abs(gl[seen] - rl[seen]) <= lb).all(), f"lse: {np.abs(gl[seen] - rl[seen]).max():.3e}"
    assert not g[~seen].any()


def attend(sca, s, tree, algo, plan=None):
    plan = plan or sca.PagedTreeAttention(s.cache(sca), s.B, s.H, tokens=s.T, keys=s.table.shape[1] * s.page, algo=algo)
    plan.o.fill_(float("nan"))
    plan.lse.fill_(float("nan"))
    o, lse = plan.attend(s.q.cuda(), s.table.cuda(), ints(s.lengths).cuda(), counts=ints(s.counts).cuda(),
                         tree=None if tree is None else tree.cuda())
    assert plan.read_status() == 0
    compare(o, lse, s, tree, plan.scale, s.dtype == torch.bfloat16 and algo != sca.capi.SCA_ALGO_SIMT)
    return plan, o, lse


ATTEND = [
    # B, Hkv, group, T, D, page, lengths, counts, tree, dtype
    (1, 1, 1, 1, 64, 16, [0], None, False, "bf16"), (1, 2, 4, 1, 128, 16, [1], None, False, "bf16"),
    (4, 2, 4, 1, 128, 64, [127, 128, 0, 129], [1, 1, 1, 0], False, "bf16"),
    (5, 1, 8, 1, 64, 32, [-3, 15, 16, 17, 500], None, False, "bf16"),
    (3, 2, 5, 24, 128, 64, [300, 0, 77], [24, 24, 3], True, "bf16"),
    (2, 1, 4, 64, 128, 128, [640, 100], [64, 33], True, "bf16"),      # two row tiles
    (2, 2, 3, 64, 64, 16, [129, 700], None, True, "bf16"),            # one and a half
    (3, 1, 6, 64, 128, 256, [1000, 255, 0], [64, 64, 64], True, "bf16"),   # three
    (6, 3, 2, 7, 64, 16, [5, 121, 122, 127, 128, 250], [7, 7, 6, 0, 1, 7], True, "bf16"),
    (4, 2, 3, 9, 128, 16, [0, 100, 119, 500], [9, 9, 5, 0], True, "bf16"), (3, 3, 4, 8, 64, 32, [250, 3, 128], None, False, "bf16"),
    (1200, 1, 2, 1, 64, 16, [(7 * i) % 45 for i in range(1200)], [int(i % 11 > 0) for i in range(1200)], False, "bf16"),
    (2, 1, 1, 16, 128, 64, [1000, 112], [16, 16], True, "bf16"), (40, 4, 4, 1, 64, 16, [(53 * i) % 700 for i in range(40)], None, False, "bf16"),
    (2, 1, 1, 300, 128, 32, [0, 77], [300, 111], False, "bf16"),      # pieces of prompts
    (1, 2, 2, 200, 64, 64, [513], None, False, "bf16"), (2, 1, 2, 700, 64, 32, [300, 0], [700, 123], False, "bf16"),
    (33, 1, 1, 270, 128, 16, [(17 * i) % 90 for i in range(33)], [270 - 8 * i for i in range(33)], False, "bf16"),
    (1, 1, 2, 1, 128, 64, [9000], None, False, "bf16"),               # one request over many SMs
    (70, 2, 2, 2, 64, 16, [(37 * i) % 400 for i in range(70)], None, True, "bf16"),
    (3, 2, 3, 9, 64, 32, [100, 31, 0], [9, 2, 9], True, "f32"), (2, 2, 4, 1, 128, 16, [1500, 3], None, False, "f32"),
    (2, 1, 2, 40, 128, 64, [200, 0], [40, 13], True, "f32"), (1, 3, 1, 150, 64, 1024, [20], None, False, "f32"),
    (4, 1, 16, 1, 64, 32, [33, 32, 31, 0], [1, 0, 1, 1], False, "f32"),
    # units in 52, 23, 10 and 6 pieces, of one row tile and of two
    (1, 1, 4, 16, 64, 128, [20000], None, True, "bf16"), (1, 1, 4, 64, 64, 64, [20000], None, True, "bf16"),
    (1, 1, 3, 64, 128, 64, [9000], None, True, "bf16"), (1, 1, 3, 20, 128, 128, [9000], None, True, "bf16"),
    (2, 8, 4, 30, 64, 64, [9000, 8000], None, True, "bf16"), (2, 6, 3, 50, 64, 32, [3000, 2000], [50, 31], True, "bf16"),
    # fp32, rows in tiles of 64: full, with a rest, one piece of the keys and many, tokens in a row
    (2, 2, 3, 41, 64, 16, [700, 0], [41, 20], True, "f32"), (3, 1, 4, 16, 128, 64, [1500, 3, 700], [16, 16, 0], True, "f32"),
    (1, 1, 1, 300, 128, 32, [250], None, False, "f32"), (1, 1, 2, 300, 64, 32, [257], [290], False, "f32"),
    (40, 4, 4, 15, 64, 128, [(53 * i) % 700 for i in range(40)], None, True, "f32"), (1, 1, 2, 64, 128, 16, [5000], None, True, "f32"),
]


def code_of(sca, algo):
    return {"auto": sca.capi.SCA_ALGO_AUTO, "simt": sca.capi.SCA_ALGO_SIMT, "tc": sca.capi.SCA_ALGO_TC}[algo]


@pytest.mark.parametrize("algo", ["auto", "simt", "tc"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(str(x) for x in c[:6]) + "-" + c[-1])
def test_attention_against_the_oracle(sca, case, algo):
    B, Hkv, group, T, D, page, lengths, counts, tree, dt = case
    if algo == "tc" and dt == "f32":
        pytest.skip("the tensor-core kernel takes bf16")
    s = Setup(B, Hkv, group, T, D, page, lengths, counts, DT[dt], seed=T + page)
    words = make_tree(B, T, seed=B + T)[0] if tree else None
    code = code_of(sca, algo)
    plan, o, lse = attend(sca, s, words, code)
    first = (o.clone(), lse.clone())
    _, o, lse = attend(sca, s, words, code, plan)
    assert torch.equal(first[0], o) and torch.equal(first[1], lse)


@pytest.mark.parametrize("algo", ["tc", "simt"])
def test_masks_that_are_no_trees(sca, algo):
    """Words that leave rows empty (also where there are no older rows), that
    see later tokens, that see all; one word list for the batch."""
    s = Setup(3, 2, 2, 10, 64, 16, [0, 40, 125], [10, 10, 10], torch.bfloat16, seed=1)
    words = torch.tensor([0, 1, 1 << 9, (1 << 10) - 1, -1, 0, 0b1010101010, 1 << 40, 3 << 8, -(1 << 63)],
                         dtype=torch.int64)
    attend(sca, s, words, code_of(sca, algo))


@pytest.mark.parametrize("algo", ["tc", "simt"])
def test_large_scores_and_one_row_that_takes_all(sca, algo):
    s = Setup(2, 2, 4, 3, 128, 32, [600, 140], None, torch.bfloat16, seed=4)
    s.q = s.q * 30
    at = s.table[0, 17].long()
    s.k[at, :, 5] = s.k[at, :, 5] * 20
    attend(sca, s, None, code_of(sca, algo))


@pytest.mark.parametrize("dt,algo", [("bf16", "tc"), ("bf16", "simt"), ("f32", "auto")])
def test_a_nan_key_shows_in_the_rows_that_see_it_and_no_others(sca, dt, algo):
    s = Setup(3, 2, 2, 4, 64, 16, [100, 30, 0], None, DT[dt], seed=6)
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1001], dtype=torch.int64)
    plan, o, lse = attend(sca, s, tree, code_of(sca, algo))
    clean = (o.clone(), lse.clone())
    for b, row, h in ((0, 57, 1), (1, 32, 0), (2, 1, 1)):   # an older row; tokens 2 and 1
        plan.cache.k[int(s.table[b, row // 16]), h, row % 16, 3] = float("nan")
    o, lse = plan.attend(s.q.cuda(), s.table.cuda(), ints(s.lengths).cuda(), tree=tree.cuda())
    hit = torch.zeros(3, 4, 4, dtype=torch.bool, device="cuda")
    hit[0, 2:] = True
    hit[1, :2, 2] = True
    hit[2, 2:, 1] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("dt,lengths", [("f32", [600, 30]), ("f32", [2500, 700]), ("bf16", [600, 30]), ("bf16", [2500, 700])])
def test_a_nan_key_among_many_rows(sca, dt, lengths):
    """64 rows a head; units in one piece and in several."""
    s = Setup(2, 2, 16, 4, 64, 16, lengths, None, DT[dt], seed=16)
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1001], dtype=torch.int64)
    plan, o, lse = attend(sca, s, tree, sca.capi.SCA_ALGO_AUTO)
    clean = (o.clone(), lse.clone())
    for b, row, h in ((0, 570, 1), (1, lengths[1] + 2, 0)):   # an older row; token 2
        plan.cache.k[int(s.table[b, row // 16]), h, row % 16, 3] = float("nan")
    o, lse = plan.attend(s.q.cuda(), s.table.cuda(), ints(s.lengths).cuda(), tree=tree.cuda())
    hit = torch.zeros(2, 32, 4, dtype=torch.bool, device="cuda")
    hit[0, 16:] = True
    hit[1, :16, 2] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("dt,algo", [("bf16", "tc"), ("bf16", "simt"), ("f32", "auto")])
def test_pools_of_other_layouts(sca, dt, algo):
    """Rows before heads, one layer of a pool of several, queries out of a wider tensor."""
    s = Setup(2, 2, 2, 3, 64, 32, [70, 200], None, DT[dt], seed=8)
    both = torch.full((s.pages, 2, 3, s.page, s.Hkv, s.D), float("nan"), dtype=s.dtype)
    both[:, 0, 1], both[:, 1, 1] = s.k.transpose(1, 2), s.v.transpose(1, 2)
    dev = both.cuda()
    pools = tuple(dev[:, i, 1].transpose(1, 2) for i in range(2))
    cache = sca.PagedKVCache(s.pages, s.Hkv, s.D, page=s.page, dtype=s.dtype, pools=pools)
    plan = sca.PagedTreeAttention(cache, s.B, s.H, tokens=s.T, keys=s.table.shape[1] * s.page, algo=code_of(sca, algo))
    wide = torch.zeros(s.B, s.H + 4, s.T, s.D, dtype=s.dtype, device="cuda")
    wide[:, :s.H] = s.q.cuda()
    table = torch.zeros(s.B, 50, dtype=torch.int32, device="cuda")
    table[:, 5:5 + s.table.shape[1]] = s.table.cuda()
    o, lse = plan.attend(wide[:, :s.H], table[:, 5:5 + s.table.shape[1]], ints(s.lengths).cuda())
    assert plan.read_status() == 0
    compare(o, lse, s, None, plan.scale, dt == "bf16")


def append_case(sca, B, Hkv, group, T, D, page, lengths, counts, dt, rd, layout, given, view):
    s = Setup(B, Hkv, group, T, D, page, lengths, counts, DT[dt], seed=T)
    angles = None if rd == 0 else sca.RotaryAngles(rd, layout=layout, scaling=("linear", 2.0))
    cache = s.cache(sca, angles=angles)
    plan = sca.PagedTreeAttention(cache, B, s.H, tokens=T, keys=s.table.shape[1] * page) if D in (64, 128) else None
    if view:   # one projection's output
        qkv = s.rnd(B, T, s.H + 2 * Hkv, D)
        q, k, v = (x.transpose(1, 2) for x in qkv.split([s.H, Hkv, Hkv], 2))
        dev = qkv.cuda()
        dq, dk, dv = (x.transpose(1, 2) for x in dev.split([s.H, Hkv, Hkv], 2))
    else:
        q, k, v = s.q, s.rnd(B, Hkv, T, D), s.rnd(B, Hkv, T, D)
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    slots = torch.tensor([[max(0, n) + t for t in range(T)] for n in lengths], dtype=torch.int32)
    pos = (slots // 2 + 1000) if given else slots
    args = (s.table.cuda(), ints(lengths).cuda())
    kw = dict(counts=None if counts is None else ints(counts).cuda(), positions=pos.cuda() if given else None)
    q1 = None
    if plan is not None:
        plan.q.fill_(float("nan"))
        q1 = plan.append(dq, dk, dv, *args, **kw)
    else:
        cache.append(dk, dv, *args, **kw)
    assert cache.read_status() == 0
    cnt = [max(0, min(T, c)) for c in s.counts]
    ones = np.zeros((B, 1, T, 0))
    cos, sin = ones, ones
    if rd:
        cos, sin = (x[:, None] for x in oracle.rotary_cos_sin(pos.numpy(), angles.frequencies))

    def bound(x, ref):
        n = cos.shape[-1]
        i = np.arange(n)
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        mag, ax = np.zeros(ref.shape), x.double().abs().numpy()
        mag[..., a] = mag[..., b] = ax[..., a] + ax[..., b]
        return mag * 6 * 2.0 ** -24 + (HALF[s.dtype] * 1.01 * np.abs(ref) * (mag > 0) if s.dtype == torch.bfloat16 else 0.0) + 1e-38

    k_ref = oracle.rotary(k, cos, sin, layout)
    kb = bound(k, k_ref)
    got_k, got_v = cache.k.double().cpu().numpy(), cache.v.cpu()
    want = oracle.paged_append(s.k.double().numpy(), k_ref, s.table, lengths, cnt)
    tol = oracle.paged_append(np.zeros(got_k.shape), kb, s.table, lengths, cnt)
    same = (got_k == want) | (np.isnan(got_k) & np.isnan(want))
    assert (same | (np.abs(got_k - want) <= tol)).all()
    want_v = oracle.paged_append(s.v.float().numpy(), v.float().numpy(), s.table, lengths, cnt)
    assert np.array_equal(got_v.float().numpy(), want_v, equal_nan=True)
    if q1 is not None:
        q_ref, live = oracle.rotary(q, cos, sin, layout), np.zeros((B, 1, T, 1))
        for b in range(B):
            live[b, :, :cnt[b]] = 1
        g = q1.double().cpu().numpy()
        assert (np.abs(g - q_ref * live) <= bound(q, q_ref)).all() and not (g * (1 - live)).any()


@pytest.mark.parametrize("case", [
    # B, Hkv, group, T, D, page, lengths, counts, dtype, rotary_dim, layout, positions given, out of one projection
    (1, 1, 1, 1, 64, 16, [0], None, "bf16", 64, "half", False, False),
    (3, 2, 4, 1, 128, 64, [63, 64, 5], None, "bf16", 128, "half", False, True),
    (4, 2, 2, 9, 128, 16, [7, 8, 0, 100], [9, 0, 3, 20], "bf16", 64, "interleaved", True, True),
    (2, 3, 1, 130, 64, 32, [1, 33], [130, 77], "f32", 32, "half", False, False),
    (2, 2, 2, 5, 64, 16, [-4, 11], [5, -1], "f32", 0, "half", False, True),
    (3, 1, 2, 4, 80, 64, [60, 61, 62], None, "bf16", 40, "half", True, False),
    (2, 1, 2, 4, 48, 16, [30, 61], [4, 2], "bf16", 6, "interleaved", False, True),
], ids=lambda c: "-".join(str(x) for x in c[:6]) + "-" + "-".join(str(x) for x in c[8:]))
def test_append_against_the_oracle(sca, case):
    append_case(sca, *case)


ACCEPT = [
    # B, Hkv, T, D, page, lengths, paths, dtype
    (1, 1, 1, 64, 16, [0], [[0]], "bf16"), (1, 2, 4, 64, 16, [14], [[1, 2, 3]], "bf16"),
    (5, 3, 9, 128, 32, [0, 31, 32, 100, 27], [[0, 1, 2, 3, 4, 5, 6, 7, 8], [8], [], [0, 3, 4, 8], [2, 3, 7]], "bf16"),
    (2, 2, 200, 64, 16, [5, 63], [list(range(100, 200)), [3 * i for i in range(66)]], "f32"),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", ACCEPT, ids=lambda c: "-".join(str(x) for x in c[:5]) + "-" + c[-1])
def test_acceptance_against_the_oracle(sca, case, in_place):
    B, Hkv, T, D, page, lengths, paths, dt = case
    s = Setup(B, Hkv, 1, T, D, page, lengths, None, DT[dt], seed=T + B)
    cache = s.cache(sca)
    plan = sca.PagedTreeAttention(cache, B, s.H, tokens=T, keys=s.table.shape[1] * page)
    path = torch.zeros(B, T, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = ints(p)
    accepted = [len(p) for p in paths]
    ln = ints(lengths).cuda()
    new = plan.accept(s.table.cuda(), ln, path.cuda(), ints(accepted).cuda(), out=ln if in_place else None)
    assert plan.read_status() == 0
    assert new.tolist() == [n + a for n, a in zip(lengths, accepted)]
    assert in_place or ln.tolist() == lengths
    for got, pool in ((cache.k, s.k), (cache.v, s.v)):
        want = oracle.paged_accept(pool.float().numpy(), s.table, lengths, path.tolist(), accepted)
        assert np.array_equal(got.float().cpu().numpy(), want, equal_nan=True)


def test_rows_without_a_place_are_left_out_and_reported(sca):
    """Tables that name pages outside the pool, or end too early: nothing is
    written elsewhere, the other requests are served, and the status says so."""
    capi = sca.capi
    for dt, algo in (("bf16", "tc"), ("bf16", "simt"), ("f32", "auto")):
        s = Setup(3, 2, 2, 4, 64, 16, [20, 30, 10], None, DT[dt], seed=3, spare=0)
        for bad in (-1, s.pages, 1 << 30):
            table = s.table.clone()
            table[1, 1] = bad       # rows 16 to 31 of request 1
            cache = s.cache(sca)
            plan = sca.PagedTreeAttention(cache, 3, s.H, tokens=4, keys=s.table.shape[1] * 16, algo=code_of(sca, algo))
            o, lse = plan.attend(s.q.cuda(), table.cuda(), ints(s.lengths).cuda())
            o, lse = o.clone(), lse.clone()
            assert capi.sca_read_status(plan.status.data_ptr(), 0) == capi.SCA_ERR_RANGE
            ok = sca.PagedTreeAttention(s.cache(sca), 3, s.H, tokens=4, keys=s.table.shape[1] * 16,
                                        algo=code_of(sca, algo))
            o2, lse2 = ok.attend(s.q.cuda(), s.table.cuda(), ints(s.lengths).cuda())
            assert torch.equal(o[[0, 2]], o2[[0, 2]]) and torch.equal(lse[[0, 2]], lse2[[0, 2]])
            assert torch.isfinite(o).all()
            # rows read as zeros: a request whose pages hold zeros there
            z = Setup(3, 2, 2, 4, 64, 16, [20, 30, 10], None, DT[dt], seed=3, spare=0)
            z.k[s.table[1, 1].long()], z.v[s.table[1, 1].long()] = 0, 0
            compare(o, lse, z, None, plan.scale, dt == "bf16")
            k, v = s.rnd(3, 2, 4, 64).cuda(), s.rnd(3, 2, 4, 64).cuda()
            before = (cache.k.clone(), cache.v.clone())
            cache.append(k, v, table.cuda(), ints(s.lengths).cuda())
            assert cache.read_status() == capi.SCA_ERR_RANGE
            want = [oracle.paged_append(p.float().cpu().numpy(), r.float().cpu().numpy(), s.table, s.lengths, [4, 0, 4])
                    for p, r in ((before[0], k), (before[1], v))]
            for b in (2, 3):   # rows 32 and 33 of request 1 have their page
                page, row = int(s.table[1, 2]), 30 + b - 32
                want[0][page, :, row], want[1][page, :, row] = k[1, :, b].float().cpu(), v[1, :, b].float().cpu()
            assert np.array_equal(cache.k.float().cpu().numpy(), want[0], equal_nan=True)
            assert np.array_equal(cache.v.float().cpu().numpy(), want[1], equal_nan=True)
        # a table that ends before the rows do
        cache = s.cache(sca)
        plan = sca.PagedTreeAttention(cache, 3, s.H, tokens=4, keys=32, algo=code_of(sca, algo))
        short = s.table[:, :2].contiguous()
        o, lse = plan.attend(s.q.cuda(), short.cuda(), ints(s.lengths).cuda())
        assert torch.isfinite(o).all()
        assert capi.sca_read_status(plan.status.data_ptr(), 0) == capi.SCA_ERR_RANGE
        before = cache.k.clone()
        cache.append(k, v, short.cuda(), ints([20, 32, 1 << 30]).cuda(), counts=ints([0, 4, 4]).cuda())
        assert cache.read_status() == capi.SCA_ERR_RANGE
        assert torch.equal(torch.nan_to_num(before), torch.nan_to_num(cache.k))


def test_paths_that_do_not_rise_leave_the_request_as_it_was(sca):
    capi = sca.capi
    s = Setup(5, 1, 1, 4, 64, 16, [3, 20, 7, 9, 2], None, torch.float32, seed=2)
    for row in ([1, 1, 2, 3], [0, 2, 1, 3], [1, 2, 3, 4], [-1, 0, 1, 2]):
        cache = s.cache(sca)
        plan = sca.PagedTreeAttention(cache, 5, 1, tokens=4, keys=s.table.shape[1] * 16)
        path = ints([[0, 2, 3, 0], row, [1, 2, 3, 0], [0, 0, 0, 0], [3, 9, 9, 9]])
        acc = [3, 4, 3, 0, 1]
        new = plan.accept(s.table.cuda(), ints(s.lengths).cuda(), path.cuda(), ints(acc).cuda())
        assert cache.read_status() == capi.SCA_ERR_RANGE
        assert new.tolist() == [6, 20, 10, 9, 3]
        acc[1] = 0
        want = oracle.paged_accept(s.k.numpy(), s.table, s.lengths, path.tolist(), acc)
        assert np.array_equal(cache.k.cpu().numpy(), want, equal_nan=True)


def test_calls_that_are_refused(sca):
    s = Setup(2, 2, 2, 3, 64, 16, [20, 5], None, torch.bfloat16, seed=1)
    cache = s.cache(sca, angles=sca.RotaryAngles(64))
    plan = sca.PagedTreeAttention(cache, 2, 4, tokens=3, keys=64)
    table, ln, q = s.table[:, :4].contiguous().cuda(), ints(s.lengths).cuda(), s.q.cuda()
    k = s.rnd(2, 2, 3, 64).cuda()
    tree = torch.ones(2, 3, dtype=torch.int64, device="cuda")
    flat = torch.zeros(2 * 4 * 3 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :2]), dict(q=q.transpose(2, 3)), dict(q=plan.o),
                dict(q=flat[4:4 + q.numel()].view_as(q)), dict(q=torch.cat([q, q], 3)[..., ::2]),
                dict(table=table.long()), dict(table=table[:1]), dict(table=table.cpu()), dict(table=table.t()),
                dict(table=torch.cat([table, table], 1)), dict(lengths=ln.long()), dict(lengths=ln[:1]),
                dict(lengths=ln.cpu()), dict(counts=ln.long()), dict(counts=ln[:1]), dict(tree=tree.int()),
                dict(tree=tree[:, :2]), dict(tree=tree.cpu()), dict(tree=tree[:1])):
        with pytest.raises(ValueError):
            plan.attend(**{**dict(q=q, table=table, lengths=ln), **bad})
    for bad in (dict(q=q[:, :2]), dict(q=plan.q), dict(k=k.float()), dict(k=k[:, :1]), dict(v=k[:1]), dict(v=k.cpu()),
                dict(k=k.transpose(2, 3)), dict(table=table.long()), dict(lengths=ln.long()), dict(counts=ln[:1]),
                dict(positions=ln), dict(positions=torch.zeros(2, 3, device="cuda"))):
        with pytest.raises(ValueError):
            plan.append(**{**dict(q=q, k=k, v=k, table=table, lengths=ln), **bad})
    path = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for bad in (dict(path=path.long()), dict(path=path[:, :2]), dict(path=path.t().contiguous().t()),
                dict(accepted=ln[:1]), dict(accepted=ln.long()), dict(out=ln.long()), dict(out=ln[:1]),
                dict(table=table[:1]), dict(lengths=ln.cpu())):
        with pytest.raises(ValueError):
            plan.accept(**{**dict(table=table, lengths=ln, path=path, accepted=ln), **bad})
    plan.attend(q, table, ln, tree=tree)
    long = sca.PagedTreeAttention(cache, 2, 4, tokens=65, keys=64)
    with pytest.raises(ValueError):
        long.attend(s.rnd(2, 4, 65, 64).cuda(), table, ln, tree=torch.ones(2, 65, dtype=torch.int64, device="cuda"))
