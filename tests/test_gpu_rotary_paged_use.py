"""Positions, cache and attention as a program uses them: a prompt trained on
and then continued, drafted tokens verified and accepted step by step, captured
steps, two plans on two streams."""
import math
import random

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sca():
    import sharded_causal_softmax_gb300 as m
    from sharded_causal_softmax_gb300 import build
    build.build()
    return m


def rnd(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def algo(sca, name):
    return {"tc": sca.capi.SCA_ALGO_TC, "simt": sca.capi.SCA_ALGO_SIMT}[name]


@pytest.mark.parametrize("dtype,page", [(torch.bfloat16, 64), (torch.float32, 16)])
def test_a_prompt_and_what_follows_it_are_one_causal_sequence(sca, dtype, page):
    """The framework's causal attention with rotary positions over S rows, and
    the same rows as a prompt in two pieces and then tokens one by one."""
    B, H, Hkv, S, D, first = 2, 4, 2, 256, 64, 100
    angles = sca.RotaryAngles(64, scaling=("base", 2.0))
    q, k, v = (rnd(B, h, S, D, seed=i, dtype=dtype) for i, h in enumerate((H, Hkv, Hkv)))
    whole = sca.ShardedCausalAttention(B, H, S, D, 1, layout="contiguous", kv_heads=Hkv, dtype=dtype, rotary=angles)
    want, lse = whole.forward(q, k, v)
    each = S // page
    cache = sca.PagedKVCache(B * each + 1, Hkv, D, page=page, dtype=dtype, angles=angles)
    table = torch.randperm(B * each + 1, device="cuda")[:B * each].to(torch.int32).view(B, each)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    piece = sca.PagedTreeAttention(cache, B, H, tokens=first, keys=S)
    one = sca.PagedTreeAttention(cache, B, H, keys=S)
    got, got_lse = torch.empty_like(want), torch.empty_like(lse)
    at = 0
    while at < S:
        plan = piece if at + first <= 2 * first else one
        rows = slice(at, at + plan.T)
        q1 = plan.append(q[:, :, rows], k[:, :, rows], v[:, :, rows], table, lengths)
        o, l = plan.attend(q1, table, lengths)
        got[:, :, rows], got_lse[:, :, rows] = o.float(), l
        lengths += plan.T
        at += plan.T
    assert piece.read_status() == 0 and one.read_status() == 0
    # both sides round P (bf16: 2^-8 of A each, |v| < 6) and this one its result; fp32: scores off by
    # D 2^-23 |q| |k| scale (|q|, |k| < 14), each way and on both sides
    err = 4 * (D * 2.0 ** -23 * 14 * 14 / math.sqrt(D) + S * 2.0 ** -23) + (3 * 2.0 ** -8 if dtype == torch.bfloat16 else 0)
    assert (got - want).abs().max().item() <= 6 * err
    assert (got_lse - lse).abs().max().item() <= 4 * D * 2.0 ** -23 * 14 * 14 / math.sqrt(D) + 1e-5


@pytest.mark.parametrize("tree_algo", ["tc", "simt"])
def test_drafts_verified_and_accepted_are_the_tokens_decoded_one_by_one(sca, tree_algo):
    """Step by step: a tree of drafts is appended at its depths, attended to,
    and a path of it kept; the kept nodes' outputs are those of plain decoding
    of that path."""
    B, H, Hkv, D, page, T, steps = 3, 4, 2, 64, 16, 7, 6
    angles = sca.RotaryAngles(32, layout="interleaved")
    rng = random.Random(1)
    start = [40, 0, 15]
    cap = max(start) + steps * T + T
    each = -(-cap // page)

    def fresh():
        cache = sca.PagedKVCache(B * each, Hkv, D, page=page, angles=angles)
        cache.k.fill_(float("nan"))
        cache.v.fill_(float("inf"))
        return cache, torch.randperm(B * each, device="cuda").to(torch.int32).view(B, each)

    drafted, plain = fresh(), fresh()
    lengths = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2)]
    prompt = [rnd(B, Hkv, max(start), D, seed=i) for i in range(2)]
    counts = torch.tensor(start, dtype=torch.int32, device="cuda")
    for (cache, table), n in zip((drafted, plain), lengths):
        cache.append(*prompt, table, n, counts=counts)
        n += counts
    tree_plan = sca.PagedTreeAttention(drafted[0], B, H, tokens=T, keys=cap, algo=algo(sca, tree_algo))
    one = sca.PagedTreeAttention(plain[0], B, H, keys=cap)
    for step in range(steps):
        words, depths, paths = [], [], []
        for b in range(B):
            w, d, ps = [], [], []
            for t in range(T):
                p = rng.randint(max(-1, t - 3), t - 1) if t else -1
                ps.append(p)
                w.append((w[p] if p >= 0 else 0) | 1 << t)
                d.append(d[p] + 1 if p >= 0 else 0)
            leaf, path = rng.randrange(T), []
            while leaf >= 0:
                path.insert(0, leaf)
                leaf = ps[leaf]
            words.append(w)
            depths.append(d)
            paths.append(path)
        q, k, v = (rnd(B, h, T, D, seed=100 * step + i) for i, h in enumerate((H, Hkv, Hkv)))
        tree = torch.tensor(words, dtype=torch.int64, device="cuda")
        pos = lengths[0][:, None] + torch.tensor(depths, dtype=torch.int32, device="cuda")
        q1 = tree_plan.append(q, k, v, drafted[1], lengths[0], positions=pos)
        o, lse = tree_plan.attend(q1, drafted[1], lengths[0], tree=tree)
        path = torch.tensor([p + [0] * (T - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        acc = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        tree_plan.accept(drafted[1], lengths[0], path, acc, out=lengths[0])
        for i in range(max(len(p) for p in paths)):
            node = [p[min(i, len(p) - 1)] for p in paths]
            live = torch.tensor([int(i < len(p)) for p in paths], dtype=torch.int32, device="cuda")
            pick = lambda x: torch.stack([x[b, :, n] for b, n in enumerate(node)])[:, :, None]
            q2 = one.append(pick(q), pick(k), pick(v), plain[1], lengths[1], counts=live)
            o2, lse2 = one.attend(q2, plain[1], lengths[1], counts=live)
            lengths[1] += live
            for b in range(B):
                if i < len(paths[b]):
                    # P rounded to bf16 on both sides (2^-8 of A each, |v| < 6), relative to different maxima, and the results
                    assert (o[b, :, node[b]].float() - o2[b, :, 0].float()).abs().max().item() <= 6 * 4 * 2.0 ** -8
                    assert (lse[b, :, node[b]] - lse2[b, :, 0]).abs().max().item() <= 1e-4
                else:
                    assert not o2[b].any() and torch.isneginf(lse2[b]).all()
        assert torch.equal(lengths[0], lengths[1])
    assert tree_plan.read_status() == 0 and one.read_status() == 0
    # the caches hold the same rows
    for b in range(B):
        at = torch.arange(int(lengths[0][b]), device="cuda")
        rows = [cache.k[table[b].long()[at // page], :, at % page] for cache, table in (drafted, plain)]
        assert torch.equal(rows[0], rows[1])


@pytest.mark.parametrize("step_algo", ["tc", "simt"])
def test_a_captured_step_is_replayed_while_the_cache_grows(sca, step_algo):
    """append, attend and the lengths in one graph: replays go on from one
    another, and equal the same calls made one by one."""
    B, H, Hkv, D, page, steps = 2, 8, 2, 128, 16, 40
    angles = sca.RotaryAngles(128)
    each = -(-(200 + steps) // page)
    table = torch.randperm(B * each, device="cuda").to(torch.int32).view(B, each)
    start = torch.tensor([200, 120], dtype=torch.int32, device="cuda")
    old = [rnd(B * each, Hkv, page, D, seed=i) for i in range(2)]
    new = [rnd(steps, B, h, 1, D, seed=5 + i) for i, h in enumerate((H, Hkv, Hkv))]

    def build(pools):
        cache = sca.PagedKVCache(B * each, Hkv, D, page=page, angles=angles, pools=pools)
        return cache, sca.PagedTreeAttention(cache, B, H, keys=each * page, algo=algo(sca, step_algo))

    outs = []
    cache, plan = build(tuple(t.clone() for t in old))
    lengths = start.clone()
    for i in range(steps):
        q1 = plan.append(*(t[i] for t in new), table, lengths)
        o, lse = plan.attend(q1, table, lengths)
        outs.append((o.clone(), lse.clone()))
        lengths += 1
    cache2, plan2 = build(tuple(t.clone() for t in old))
    now = [t[0].clone() for t in new]
    lengths2 = start.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # a first call outside the capture; its row is written again below
        plan2.attend(plan2.append(*now, table, lengths2), table, lengths2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = plan2.attend(plan2.append(*now, table, lengths2), table, lengths2)
        lengths2 += 1
    for i in range(steps):
        for to, t in zip(now, new):
            to.copy_(t[i])
        graph.replay()
        assert torch.equal(o, outs[i][0]) and torch.equal(lse, outs[i][1]), i
    assert torch.equal(cache.k, cache2.k) and torch.equal(cache.v, cache2.v) and torch.equal(lengths, lengths2)
    assert plan.read_status() == 0 and plan2.read_status() == 0


@pytest.mark.parametrize("both", ["tc", "simt"])
def test_two_plans_on_two_streams(sca, both):
    B, H, Hkv, D, page, n = 8, 8, 2, 128, 64, 1500
    each = -(-(n + 4) // page)
    made = []
    for i in range(2):
        pools = tuple(rnd(B * each, Hkv, page, D, seed=10 * i + j) for j in range(2))
        cache = sca.PagedKVCache(B * each, Hkv, D, page=page, pools=pools)
        plan = sca.PagedTreeAttention(cache, B, H, tokens=4, keys=each * page, algo=algo(sca, both))
        table = torch.randperm(B * each, device="cuda").to(torch.int32).view(B, each)
        lengths = torch.randint(0, n, (B,), device="cuda").to(torch.int32)
        made.append((plan, rnd(B, H, 4, D, seed=20 + i), table, lengths))
    want = [tuple(t.clone() for t in plan.attend(q, table, lengths)) for plan, q, table, lengths in made]
    streams = [torch.cuda.Stream() for _ in made]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, (plan, q, table, lengths) in zip(streams, made):
            with torch.cuda.stream(s):
                plan.attend(q, table, lengths)
    torch.cuda.synchronize()
    for (o, lse), (plan, *_rest) in zip(want, made):
        assert torch.equal(plan.o, o) and torch.equal(plan.lse, lse) and plan.read_status() == 0


@pytest.mark.parametrize("group", [2, 5])
def test_two_graphs_of_one_plan_and_lengths_that_change(sca, group):
    """Drafted trees of 12 tokens (24 and 60 query rows; units cut over several
    SMs) captured twice and replayed in turn while the lengths change: the
    counters that cut units are joined by come back to zero every time."""
    B, Hkv, T, D, page, n = 3, 2, 12, 64, 32, 9000
    H, each = Hkv * group, -(-(n + T) // page)
    pools = tuple(rnd(B * each, Hkv, page, D, seed=j) for j in range(2))
    cache = sca.PagedKVCache(B * each, Hkv, D, page=page, pools=pools)
    table = torch.randperm(B * each, device="cuda").to(torch.int32).view(B, each)
    make = lambda: sca.PagedTreeAttention(cache, B, H, tokens=T, keys=each * page, algo=sca.capi.SCA_ALGO_TC)
    plan, eager = make(), make()
    tree = torch.tensor([(1 << t) | 1 for t in range(T)], dtype=torch.int64, device="cuda")
    q = [rnd(B, H, T, D, seed=7 + i) for i in range(2)]
    lengths, counts = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.attend(q[0], table, lengths, counts=counts, tree=tree)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan.attend(x, table, lengths, counts=counts, tree=tree)
        graphs.append(g)
    for ln, ct in (([n, 0, 500], [12, 12, 0]), ([3000, 8999, 8000], [12, 1, 7]), ([0, 0, 0], [0, 0, 0]), ([n, n, n], [12, 12, 12])):
        lengths.copy_(torch.tensor(ln, dtype=torch.int32))
        counts.copy_(torch.tensor(ct, dtype=torch.int32))
        for g, x in zip(graphs, q):
            g.replay()
            got = (plan.o.clone(), plan.lse.clone())
            o, lse = eager.attend(x, table, lengths, counts=counts, tree=tree)
            assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    assert plan.read_status() == 0 and eager.read_status() == 0


@pytest.mark.parametrize("dtype,algo_name,T", [(torch.bfloat16, "tc", 1), (torch.bfloat16, "tc", 20),
                                               (torch.bfloat16, "simt", 2), (torch.float32, "simt", 3),
                                               (torch.float32, "simt", 20)])
def test_offsets_beyond_32_bits(sca, dtype, algo_name, T):
    """Pages and heads that lie 2^31 elements apart and more."""
    Hkv, group, D, page, n = 2, 2, 64, 16, 100
    far = (1 << 31) + 4096
    pages = 2
    base = [torch.empty(far + (1 << 20) * pages + page * D * 4, dtype=dtype, device="cuda") for _ in range(2)]
    # heads far apart, pages 2^20 elements
    pools = tuple(b.as_strided((pages, Hkv, page, D), (1 << 20, far, D, 1)) for b in base)
    ref = []
    for i, p in enumerate(pools):
        x = rnd(pages, Hkv, page, D, seed=i, dtype=dtype)
        p.copy_(x)
        ref.append(x)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([2 * page - T - 1], dtype=torch.int32, device="cuda") if T < page else \
        torch.tensor([2], dtype=torch.int32, device="cuda")
    q = rnd(1, Hkv * group, T, D, seed=5, dtype=dtype)
    k, v = rnd(1, Hkv, T, D, seed=6, dtype=dtype), rnd(1, Hkv, T, D, seed=7, dtype=dtype)
    outs = []
    for ps in (pools, tuple(ref)):
        cache = sca.PagedKVCache(pages, Hkv, D, page=page, dtype=dtype, pools=ps, angles=sca.RotaryAngles(64))
        plan = sca.PagedTreeAttention(cache, 1, Hkv * group, tokens=T, keys=2 * page, algo=algo(sca, algo_name))
        q1 = plan.append(q, k, v, table, lengths)
        o, lse = plan.attend(q1, table, lengths)
        acc = torch.tensor([1], dtype=torch.int32, device="cuda")
        path = torch.zeros(1, T, dtype=torch.int32, device="cuda")
        path[0, 0] = T - 1
        new = plan.accept(table, lengths, path, acc)
        assert plan.read_status() == 0
        outs.append((o.clone(), lse.clone(), new.clone(), cache.k.contiguous(), cache.v.contiguous()))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    # rows of a tensor whose heads are as far apart, turned
    plan = sca.RotaryPositions(1, 2, 3, D, sca.RotaryAngles(64), dtype=dtype)
    x = base[0].as_strided((1, 2, 3, D), (0, far, D, 1))
    a, b = (t.clone() for t in plan.forward(x, x.contiguous()))
    assert torch.equal(a, b)


def test_another_stream_than_the_tensors(sca):
    """Calls on a side stream that waits for the tensors' own, and events back."""
    B, H, Hkv, D, page = 2, 4, 2, 64, 16
    cache = sca.PagedKVCache(20, Hkv, D, page=page, angles=sca.RotaryAngles(64))
    cache.k.zero_(), cache.v.zero_()
    plan = sca.PagedTreeAttention(cache, B, H, keys=160)
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = [tuple(rnd(B, h, 1, D, seed=10 * i + j) for j, h in enumerate((H, Hkv, Hkv))) for i in range(30)]
    want = []
    for x in rows:
        want.append(plan.attend(plan.append(*x, table, lengths), table, lengths)[0].clone())
        lengths += 1
    cache.k.zero_(), cache.v.zero_()
    lengths.zero_()
    side = torch.cuda.Stream()
    got = []
    for i, x in enumerate(rows):
        s = side if i % 2 else torch.cuda.current_stream()
        other = torch.cuda.current_stream() if i % 2 else side
        s.wait_stream(other)
        with torch.cuda.stream(s):
            got.append(plan.attend(plan.append(*x, table, lengths), table, lengths)[0].clone())
            lengths += 1
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and plan.read_status() == 0


@pytest.mark.parametrize("T,short", [(1, 2000), (12, 150)])
def test_short_and_long_tables_of_one_plan(sca, T, short):
    """The kernel is chosen by the table that a call brings: of a plan for long
    tables, short ones go to fp32 arithmetic, whose partials must leave the
    counters of the tensor-core kernels alone."""
    B, Hkv, group, D, page, n = 2, 2, 2, 64, 16, 1000
    H, each = Hkv * group, 6000 if T == 1 else 2000
    pools = tuple(rnd(2 * n, Hkv, page, D, seed=j) for j in range(2))
    cache = sca.PagedKVCache(2 * n, Hkv, D, page=page, pools=pools)
    table = torch.arange(2 * n, device="cuda").to(torch.int32).repeat(1, each // (2 * n) + 1)[:, :each].repeat(2, 1)
    table = table.contiguous()
    q = rnd(B, H, T, D, seed=9)
    make = lambda: sca.PagedTreeAttention(cache, B, H, tokens=T, keys=each * page)
    plan = make()
    for few in (each, short, each, 64, short, each):
        lengths = torch.tensor([few * page - T, few * page // 2], dtype=torch.int32, device="cuda")
        o, lse = (t.clone() for t in plan.attend(q, table[:, :few], lengths))
        fresh = make()
        o2, lse2 = fresh.attend(q, table[:, :few], lengths)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert plan.read_status() == 0
    assert not plan._ws[:1024].any()
