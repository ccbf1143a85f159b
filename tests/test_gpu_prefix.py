"""GPU parity of decode attention over a shared prefix against the fp64
oracle.

Bounds: o = sum_j p_j v_j / sum_j p_j with A = sum_j p_j |v_j| / sum_j p_j.
The tensor-core kernel rounds each p_j to bf16 for the product with V (half a
step, 2^-8 of A at most); scores are fp32 sums of exact products, and a score
that is off by e changes its weight by e: D 2^-23 sum_d |q_d k_d| scale, which
is below 2^-16 x (|s| summed by magnitude) here and is written out below; fp32
sums over n keys add n 2^-24 of A (the tensor cores' truncation twice that).
The output adds half a step of its type.  lse is a log: the absolute error is
the relative one of the sum, plus half a step of itself."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def sca():
    import sharded_causal_softmax_gb300 as m
    from sharded_causal_softmax_gb300 import build
    build.build()
    return m


def make(B, Hkv, group, T, prefix, cap, D, dtype, lengths, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype)
    q = rnd(B, Hkv * group, T, D)
    kp, vp = (rnd(Hkv, prefix, D), rnd(Hkv, prefix, D)) if prefix else (None, None)
    ks, vs = (rnd(B, Hkv, cap, D), rnd(B, Hkv, cap, D)) if cap else (None, None)
    if cap:
        for b, n in enumerate(lengths):   # a cache's unwritten rows
            ks[b, :, max(0, n):] = float("nan")
            vs[b, :, max(0, n):] = float("inf")
    return q, kp, vp, ks, vs


def check(sca, plan, args, lengths, dtype, tc):
    q, kp, vp, ks, vs = args
    dev = [None if t is None else t.cuda() for t in args]
    ln = None if ks is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    plan.o.fill_(float("nan"))
    plan.lse.fill_(float("nan"))
    plan._ws.fill_(float("nan"))
    o, lse = plan.decode(*dev, ln)
    assert plan.read_status() == 0
    compare(plan, o, lse, args, lengths, dtype, tc)
    return o, lse


def compare(plan, o, lse, args, lengths, dtype, tc):
    q, kp, vp, ks, vs = args
    ref, rl, mag = oracle.prefix_decode(q, kp, vp, ks, vs, lengths, plan.scale)
    n = (0 if kp is None else kp.shape[1]) + (0 if ks is None else max([0] + [int(x) for x in lengths]))
    # scores: sum_d |q_d k_d| <= |q| |k| (2-norms); a weight moves by that error, each way
    kmax = max(float(torch.nan_to_num(t.double(), nan=0.0).norm(dim=-1).max()) for t in (kp, ks)
               if t is not None and t.numel())
    es = plan.D * 2.0 ** -23 * float(q.double().norm(dim=-1).max()) * kmax * abs(plan.scale) + 2.0 ** -21
    err = 2 * es + n * 2.0 ** -23 + 2.0 ** -20 + (2.0 ** -8 if tc else 0.0)
    g, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl)) and np.isfinite(g).all()
    bound = HALF[dtype] * 1.01 * np.abs(ref) + err * mag
    assert (np.abs(g - ref) <= bound).all(), f"o: worst {(np.abs(g - ref) / np.maximum(bound, 1e-37)).max():.2f} of the bound"
    seen = ~np.isneginf(rl)
    d = np.abs(gl[seen] - rl[seen])
    lb = es + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * np.abs(rl[seen])
    assert (d <= lb).all(), f"lse: {d.max():.3e}"
    assert not g[~seen].any()
    return ref


CASES = [
    # B, Hkv, group, T, prefix, cap, D, dtype, lengths
    (1, 1, 1, 1, 1, 1, 64, "bf16", [1]), (1, 1, 1, 1, 1, 0, 128, "bf16", None), (2, 2, 1, 1, 0, 5, 64, "bf16", [5, 0]),
    (3, 2, 4, 1, 127, 130, 128, "bf16", [130, 1, 128]), (5, 1, 8, 1, 128, 64, 64, "bf16", [64, 0, 3, 63, -1]),
    (13, 2, 5, 3, 700, 300, 128, "bf16", [3, 2, 1, 0, 300, 299, 256, 257, 128, 129, 127, 5, 4]),
    (33, 1, 7, 2, 1000, 40, 64, "bf16", [7 + i % 33 for i in range(33)]),
    (2, 1, 128, 1, 300, 200, 128, "bf16", [200, 33]), (3, 1, 65, 1, 129, 100, 128, "bf16", [99, 100, 1]),
    (3, 2, 16, 8, 257, 20, 64, "bf16", [8, 20, 9]), (1, 2, 2, 1, 5000, 0, 128, "bf16", None),
    (4, 3, 1, 1, 0, 2000, 128, "bf16", [2000, 1999, 1, 0]),
    # rows so many that several are joined by one CTA, also a number that four does not divide
    (40, 4, 3, 1, 300, 0, 64, "bf16", None), (20, 2, 5, 3, 200, 0, 128, "bf16", None),
    (130, 3, 5, 1, 200, 130, 128, "bf16", [(i * 37) % 131 for i in range(130)]),
    (150, 4, 2, 1, 100, 140, 64, "bf16", [(i * 53) % 141 for i in range(150)]),
    (3, 2, 3, 2, 100, 70, 64, "f32", [70, 1, 33]), (2, 2, 4, 1, 1500, 513, 128, "f32", [513, 512]),
    (1, 1, 33, 1, 33, 31, 64, "f32", [31]),
]


@pytest.mark.parametrize("algo", ["auto", "simt"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:8]))
def test_against_the_oracle(sca, case, algo):
    B, Hkv, group, T, prefix, cap, D, dt, lengths = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    args = make(B, Hkv, group, T, prefix, cap, D, dtype, lengths, seed=prefix + cap)
    plan = sca.SharedPrefixAttention(B, Hkv * group, D, prefix, cap, kv_heads=Hkv, tokens=T, dtype=dtype,
                                     algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    o, lse = check(sca, plan, args, lengths, dtype, dt == "bf16" and algo == "auto")
    a = (o.clone(), lse.clone())
    b = check(sca, plan, args, lengths, dtype, dt == "bf16" and algo == "auto")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("algo", ["auto", "simt"])
def test_large_scores_and_one_key_that_takes_all(sca, algo):
    B, Hkv, group, D = 2, 2, 4, 128
    args = list(make(B, Hkv, group, 1, 600, 300, D, torch.bfloat16, [300, 140], seed=4))
    args[0] = args[0] * 30
    args[1][:, 555] = args[1][:, 555] * 20
    plan = sca.SharedPrefixAttention(B, Hkv * group, D, 600, 300, kv_heads=Hkv,
                                     algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    check(sca, plan, args, [300, 140], torch.bfloat16, algo == "auto")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views(sca, dtype):
    """Caches laid out rows first, a longer prefix cache of which a part is
    used, queries out of a wider row."""
    B, Hkv, group, T, D, n, cap = 3, 2, 4, 1, 64, 200, 90
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype)
    wide = rnd(B, Hkv * group + 2 * Hkv, T, D)
    pre = rnd(2, 1000, Hkv, D)
    suf = rnd(B, cap, 2, Hkv, D)
    lengths = [90, 17, 1]

    def views(wide, pre, suf):
        return (wide[:, :Hkv * group], *(pre[i, :n].transpose(0, 1) for i in range(2)),
                *(suf[:, :, i].transpose(1, 2) for i in range(2)))

    plan = sca.SharedPrefixAttention(B, Hkv * group, D, 1000, cap, kv_heads=Hkv, dtype=dtype)
    o, lse = plan.decode(*views(wide.cuda(), pre.cuda(), suf.cuda()),
                         torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    compare(plan, o, lse, views(wide, pre, suf), lengths, dtype, dtype == torch.bfloat16)


def test_captured_with_growing_suffixes(sca):
    """A captured step is replayed while tokens are appended to the caches."""
    B, Hkv, group, D, cap = 3, 2, 4, 128, 300
    q, kp, vp, ks, vs = make(B, Hkv, group, 1, 400, cap, D, torch.bfloat16, [cap] * B, seed=8)
    dev = [t.cuda() for t in (q, kp, vp, ks, vs)]
    ln = torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda")
    plan = sca.SharedPrefixAttention(B, Hkv * group, D, 400, cap, kv_heads=Hkv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.decode(*dev, ln)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = plan.decode(*dev, ln)
    for lengths in ([1, 127, 299], [300, 128, 0], [129, 255, 256]):
        ln.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        compare(plan, o, lse, (q, kp, vp, ks, vs), lengths, torch.bfloat16, True)
    assert plan.read_status() == 0


def test_a_batch_behind_one_prefix_is_attention_over_the_whole(sca):
    """Used together: the prefix's and the requests' keys as one causal
    sequence each, whose last rows the framework's own attention computes."""
    B, H, Hkv, D, n, own = 2, 8, 4, 128, 256, 128
    q, kp, vp, ks, vs = make(B, Hkv, H // Hkv, 1, n, own, D, torch.bfloat16, [own] * B, seed=6)
    dev = [t.cuda() for t in (q, kp, vp, ks, vs)]
    plan = sca.SharedPrefixAttention(B, H, D, n, own, kv_heads=Hkv)
    o, lse = plan.decode(*dev, torch.full((B,), own, dtype=torch.int32, device="cuda"))
    whole = sca.ShardedCausalAttention(B, H, n + own, D, 1, layout="contiguous", kv_heads=Hkv)
    qq = torch.zeros(B, H, n + own, D, dtype=torch.bfloat16, device="cuda")
    qq[:, :, -1:] = dev[0]
    k, v = (torch.cat([p.expand(B, Hkv, n, D), s], 2).contiguous() for p, s in ((dev[1], dev[3]), (dev[2], dev[4])))
    wo, wl = whole.forward(qq, k, v)
    compare(plan, o, lse, (q, kp, vp, ks, vs), [own] * B, torch.bfloat16, True)
    # both sides round P (2^-8 of A each) and this one its result
    a = oracle.prefix_decode(q, kp, vp, ks, vs, [own] * B, plan.scale)[2]
    assert ((o.double() - wo[:, :, -1:].double()).abs().cpu().numpy() <= 3.1 * 2.0 ** -8 * a).all()
    assert (lse - wl[:, :, -1:]).abs().max().item() <= 1e-4


@pytest.mark.parametrize("dtype,algo", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_a_nan_key_shows_in_the_rows_that_see_it_and_no_others(sca, dtype, algo):
    """Not dropped with the pieces that have nothing: prefix key 300 of head 0
    and suffix key 5 of request 1, head 1; a key behind a length is not seen."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, Hkv, group, D, n, cap, lengths = 3, 2, 4, 64, 1000, 400, [400, 6, 5]
    q, kp, vp, ks, vs = (t.cuda() for t in make(B, Hkv, group, 1, n, cap, D, dt, [cap] * B, seed=3))
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    plan = sca.SharedPrefixAttention(B, Hkv * group, D, n, cap, kv_heads=Hkv, dtype=dt,
                                     algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    clean = [t.clone() for t in plan.decode(q, kp, vp, ks, vs, ln)]
    kp[0, 300, 7] = float("nan")
    ks[1:, 1, 5, 3] = float("nan")   # request 1 sees it, request 2 ends before it
    o, lse = plan.decode(q, kp, vp, ks, vs, ln)
    hit = torch.zeros(B, Hkv * group, dtype=torch.bool, device="cuda")
    hit[:, :group] = True
    hit[1, group:] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["rising", "falling", "steps"])
def test_row_maxima_that_move(sca, D, order):
    """Scores that grow by hundreds along the keys (every group of 32 raises
    the maximum), fall, or jump within a tile."""
    B, Hkv, group, n, cap = 2, 2, 3, 640, 200
    g = torch.Generator().manual_seed(9)
    q, kp, vp, ks, vs = make(B, Hkv, group, 1, n, cap, D, torch.bfloat16, [200, 77], seed=12)
    j = torch.arange(n + cap, dtype=torch.float32)
    size = {"rising": j / (n + cap), "falling": 1 - j / (n + cap), "steps": (j % 96 < 16).float()}[order]
    u = torch.nn.functional.normalize(torch.randn(D, generator=g), dim=0)
    q = (q + 3 * math.sqrt(D) * u).bfloat16()                       # every query leans on u
    kp = (0.1 * kp + (12 * size[:n] * math.sqrt(D))[:, None] * u).bfloat16()
    ks = (0.1 * ks + (12 * size[n:] * math.sqrt(D))[:, None] * u).bfloat16()
    plan = sca.SharedPrefixAttention(B, Hkv * group, D, n, cap, kv_heads=Hkv)
    check(sca, plan, (q, kp, vp, ks, vs), [200, 77], torch.bfloat16, True)
