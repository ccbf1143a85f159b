"""Decaying linear attention and shared-prefix decoding as a program uses
them: calls that the plans refuse, broadcast and far-apart tensors, two plans
on two streams, a chain of both operators with no synchronisation between."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sca():
    import sharded_causal_softmax_gb300 as m
    from sharded_causal_softmax_gb300 import build
    build.build()
    return m


def rnd(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


DECAY = [-0.3, -0.05, -0.004]


def test_decay_plan_calls_that_are_refused(sca):
    B, H, S, D = 2, 3, 40, 64
    plan = sca.DecayLinearAttention(B, H, S, D, DECAY, backward=True)
    q, k, v, do = (rnd(B, H, S, D, seed=i) for i in range(4))
    s = rnd(B, H, D, D, dtype=torch.float32)
    ln = torch.tensor([40, 7], dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError):
        plan.backward(do)
    o, _ = plan.forward(q, k, v, state=s, lengths=ln)
    flat = torch.zeros(B * H * S * D + 8, dtype=torch.bfloat16, device="cuda")
    bad_rows = [q.float(), q.cpu(), q[:1], q[:, :2], q[..., :32], rnd(B, H, S + 1, D), rnd(B, H, D), q.transpose(2, 3),
                rnd(B, H, D, S).transpose(2, 3), rnd(B, H, S, D + 4)[..., :D], q[:, :, :1].expand(B, H, S, D),
                flat[4:4 + q.numel()].view_as(q), o]
    for t in bad_rows:
        for i in range(3):
            args = [q, k, v]
            args[i] = t
            with pytest.raises(ValueError):
                plan.forward(*args)
    for t in (s.half(), s[:1], s.cpu(), s.transpose(2, 3), s[..., :32], plan.state, s.transpose(0, 1),
              s[:, :1].expand(B, H, D, D)):
        with pytest.raises(ValueError):
            plan.forward(q, k, v, state=t)
    for t in (ln.long(), ln.cpu(), ln[:1], torch.zeros(4, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            plan.forward(q, k, v, lengths=t)
    plan.forward(q, k, v, state=s, lengths=ln)
    for t in bad_rows[:-1] + [do[:, :, :20], plan.forward(q, k, v, state=s, lengths=ln)[0]]:
        with pytest.raises(ValueError):
            plan.backward(t)
    with pytest.raises(ValueError):
        plan.backward(do, dstate=s[:1])
    first = plan.backward(do, dstate=s)[3]
    with pytest.raises(ValueError):
        plan.backward(do, dstate=first)
    one = [t[:, :, 0] for t in (q, k, v)]
    with pytest.raises(ValueError):
        plan.step(*one, s[:1].expand(B, H, D, D))
    with pytest.raises(ValueError):
        plan.step(one[0].float(), *one[1:], s)
    with pytest.raises(ValueError):
        plan.step(plan.step(*one, s.clone()), *one[1:], s)
    with pytest.raises(RuntimeError):
        sca.DecayLinearAttention(B, H, S, D, DECAY).backward(do)
    # a plan without backward: its own states only as they are
    serve = sca.DecayLinearAttention(B, H, S, D, DECAY)
    serve.forward(q, k, v)
    with pytest.raises(sca.ScaError):
        serve.forward(q, k, v, state=serve.state[:1].expand(B, H, D, D))
    serve.forward(q, k, v, state=serve.state)
    assert plan.read_status() == 0 and serve.read_status() == 0


def test_prefix_plan_calls_that_are_refused(sca):
    B, H, Hkv, T, D, n, cap = 2, 8, 2, 2, 64, 100, 50
    plan = sca.SharedPrefixAttention(B, H, D, n, cap, kv_heads=Hkv, tokens=T)
    q, p, s = rnd(B, H, T, D), rnd(Hkv, n, D), rnd(B, Hkv, cap, D)
    ln = torch.tensor([50, 20], dtype=torch.int32, device="cuda")
    o, _ = plan.decode(q, p, p, s, s, ln)
    flat = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    for t in (q.float(), q[:1], q[:, :4], q.transpose(1, 2), flat[4:4 + q.numel()].view_as(q), q[:1].expand(B, H, T, D),
              q.cpu(), o):
        with pytest.raises(ValueError):
            plan.decode(t, p, p, s, s, ln)
    for t in (None, p.float(), p[:1], rnd(Hkv, n + 1, D), p.cpu(), rnd(n, Hkv, D).transpose(0, 1), p[..., :32],
              p[:, :1].expand(Hkv, n, D), p[:, :50]):
        with pytest.raises(ValueError):
            plan.decode(q, p, t, s, s, ln)
    for t in (None, s.float(), s[:1], rnd(B, Hkv, cap + 1, D), s.cpu(), rnd(B, cap, Hkv, D).transpose(1, 2)):
        with pytest.raises(ValueError):
            plan.decode(q, p, p, s, t, ln)
    for t in (None, ln.long(), ln.cpu(), ln[:1], torch.zeros(4, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            plan.decode(q, p, p, s, s, t)
    assert plan.read_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_broadcast_inputs_are_their_copies(sca, dtype):
    """Strides of zero: one key head for all heads, one query for the batch,
    caches that heads or requests share."""
    B, H, S, D = 2, 3, 333, 64
    q, k, v = (rnd(*s, seed=i, dtype=dtype) for i, s in enumerate(((1, H, S, D), (B, 1, S, D), (1, 1, S, D))))
    do = rnd(B, 1, S, D, seed=7, dtype=dtype)
    wide = [t.expand(B, H, S, D) for t in (q, k, v, do)]
    plan = sca.DecayLinearAttention(B, H, S, D, DECAY, dtype=dtype, backward=True)
    outs = []
    for x in (wide, [t.contiguous() for t in wide]):
        o, end = plan.forward(*x[:3])
        outs.append([t.clone() for t in (o, end, *plan.backward(x[3])[:3])])
        state = rnd(B, H, D, D, seed=9, dtype=torch.float32)
        outs[-1] += [plan.step(*(t[:, :, 5] for t in x[:3]), state).clone(), state]
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    pre, suf = rnd(1, 200, D, seed=1, dtype=dtype), rnd(1, 1, 150, D, seed=2, dtype=dtype)
    ln = torch.tensor([150, 33], dtype=torch.int32, device="cuda")
    dec = sca.SharedPrefixAttention(B, 6, D, 200, 150, kv_heads=2, dtype=dtype)
    qd, got = rnd(B, 6, 1, D, seed=3, dtype=dtype), []
    for f in (lambda t: t, lambda t: t.contiguous()):
        p, s = f(pre.expand(2, 200, D)), f(suf.expand(B, 2, 150, D))
        got.append([t.clone() for t in dec.decode(qd, p, p, s, s, ln)])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert plan.read_status() == 0 and dec.read_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_far_apart(sca, dtype):
    """Views whose offsets pass 2^31 elements and 2^32 bytes give what their
    copies give."""
    S, D, far = 300, 64, 1 << 23        # 300 rows 2^23 elements apart
    buf = torch.empty((S - 1) * far + 4 * D, dtype=dtype, device="cuda")
    x = [buf[i * D:].as_strided((1, 1, S, D), (0, 0, far, 1)) for i in range(4)]
    near = [rnd(1, 1, S, D, seed=i, dtype=dtype) for i in range(4)]
    for a, b in zip(x, near):
        a.copy_(b)
    plan = sca.DecayLinearAttention(1, 1, S, D, [-0.02], dtype=dtype, backward=True)
    outs = []
    for t in (x, near):
        o, end = plan.forward(*t[:3])
        outs.append([y.clone() for y in (o, end, *plan.backward(t[3])[:3])])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    dec = sca.SharedPrefixAttention(1, 1, D, S, S, dtype=dtype)
    ln, qd, got = torch.tensor([S], dtype=torch.int32, device="cuda"), rnd(1, 1, 1, D, seed=8, dtype=dtype), []
    for t in (x, near):
        got.append([y.clone() for y in dec.decode(qd, t[0][0], t[1][0], t[2], t[3], ln)])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    # states of a step, far apart as well
    sbuf = torch.empty((1 << 31) + D * D, dtype=torch.float32, device="cuda")
    far_s = sbuf.as_strided((3, 1, D, D), (1 << 30, D * D, D, 1))
    s = rnd(3, 1, D, D, seed=4, dtype=torch.float32)
    far_s.copy_(s)
    st = sca.DecayLinearAttention(3, 1, 1, D, [-0.02], dtype=dtype)
    tok = [rnd(3, 1, D, seed=i, dtype=dtype) for i in range(3)]
    a = st.step(*tok, far_s).clone()
    assert torch.equal(a, st.step(*tok, s)) and torch.equal(far_s, s)


def test_more_than_2_to_the_31_elements(sca):
    """The last of many heads, and the last keys of a long cache, against the
    fp32 kernels on them alone.  Both round o (2^-8 of it each), and the
    tensor cores the masked product and the state's copy: 2^-8 of the sums
    over the magnitudes, as everywhere."""
    H, S, D = 18, 1 << 20, 128
    decay = torch.linspace(-0.5, -0.01, H)
    q, k, v = (torch.randn(1, H, S, D, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    o, end = sca.DecayLinearAttention(1, H, S, D, decay).forward(q, k, v)
    last = sca.DecayLinearAttention(1, 1, S, D, decay[-1:], algo=sca.capi.SCA_ALGO_SIMT)
    x = [t[:, -1:] for t in (q, k, v)]
    ro, rs = (t.clone() for t in last.forward(*x))
    mo, ms = last.forward(*(t.abs() for t in x))
    tail = slice(S - 4096, S)
    d = (o[:, -1:, tail].double() - ro[:, :, tail].double()).abs()
    # 1.05: the magnitudes' sum is itself rounded to bf16 (2^-8), and fp32 sums over what the decay leaves
    # of the rows (e^-41 after 4096) pass some 530 roundings of 2^-23: 1.6% of 2^-8
    assert (d <= 1.05 * 2.0 ** -8 * (2 * ro[:, :, tail].double().abs() + mo[:, :, tail].double())).all()
    assert ((end[:, -1:].double() - rs.double()).abs() <= 1e-4 * ms.double()).all()
    del q, k, v, o, x
    Hkv, n = 12, 1 << 21
    kp, vp = (torch.randn(Hkv, n, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    qd = rnd(1, Hkv, 1, D, seed=2)
    at = [n - 1 - 3 * h for h in range(Hkv)]
    for h in range(Hkv):   # scores of about 90 against 6 at most: all other weights together are below e^-60
        kp[h, at[h]] = 8 * qd[0, h, 0]
    dec = sca.SharedPrefixAttention(1, Hkv, D, n, 0)
    od, lse = dec.decode(qd, kp, vp, None, None, None)
    for h in range(Hkv):
        assert torch.equal(od[0, h, 0], vp[h, at[h]])
        s = dec.scale * float((qd[0, h, 0].double() * kp[h, at[h]].double()).sum())
        assert abs(float(lse[0, h, 0]) - s) <= 1e-4 * s
    assert dec.read_status() == 0


def test_plans_side_by_side_on_two_streams(sca):
    """Each with its own buffers, eager and as two captured graphs."""
    B, H, S, D = 1, 3, 3000, 128
    sides = []
    for i in range(2):
        x = [rnd(B, H, S, D, seed=10 * i + j) for j in range(4)]
        cache = [rnd(4, 2000, D, seed=50 + i), rnd(3, 4, 200, D, seed=60 + i)]
        sides.append((torch.cuda.Stream(), sca.DecayLinearAttention(B, H, S, D, DECAY, backward=True),
                      sca.SharedPrefixAttention(3, 16, D, 2000, 200, kv_heads=4), x, rnd(3, 16, 1, D, seed=70 + i), cache,
                      torch.tensor([200, 100 + i, 3], dtype=torch.int32, device="cuda")))

    def run(side):
        _, plan, dec, x, qd, (p, s), ln = side
        o, end = plan.forward(*x[:3])
        return (o, end, *plan.backward(x[3])[:3], *dec.decode(qd, p, p, s, s, ln))

    alone = []
    for side in sides:
        alone.append([t.clone() for t in run(side)])
        torch.cuda.synchronize()
    for _ in range(5):
        for side in sides:
            with torch.cuda.stream(side[0]):
                run(side)
    torch.cuda.synchronize()
    for side, want in zip(sides, alone):
        assert all(torch.equal(a, b) for a, b in zip(run(side), want))
    graphs = []
    for side in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run(side)
        graphs.append((g, outs))
        torch.cuda.synchronize()
    for _ in range(5):
        for side, (g, _) in zip(sides, graphs):
            with torch.cuda.stream(side[0]):
                g.replay()
    torch.cuda.synchronize()
    for (_, outs), want in zip(graphs, alone):
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layers_of_both_kinds_in_a_row(sca, dtype):
    """A token through layers of both kinds, each reading the one before's
    output where it lies, captured: the same bits as with a synchronisation
    after every call.  The suffixes grow with every token."""
    B, H, Hkv, D, n, cap, tokens = 5, 8, 2, 128, 700, 64, 6
    lin = [sca.DecayLinearAttention(B, H, 1, D, [-0.1] * H, dtype=dtype) for _ in range(3)]
    att = [sca.SharedPrefixAttention(B, H, D, n, cap, kv_heads=Hkv, dtype=dtype) for _ in range(3)]
    pre = [rnd(2, Hkv, n, D, seed=i, dtype=dtype) for i in range(3)]
    k, v = (rnd(B, H, D, seed=20 + i, dtype=dtype) for i in range(2))
    x0 = rnd(B, H, D, seed=30, dtype=dtype)

    def start():
        return ([rnd(B, H, D, D, seed=40 + i, dtype=torch.float32) for i in range(3)],
                [torch.zeros(2, B, Hkv, cap, D, dtype=dtype, device="cuda") for _ in range(3)],
                torch.zeros(B, dtype=torch.int32, device="cuda"), x0.clone())

    def token(states, suffix, ln, x, sync):
        ln.add_(1)
        rows = torch.arange(B, device="cuda")
        y = x
        for i in range(3):
            y = lin[i].step(y, k, v, states[i])
            if sync:
                torch.cuda.synchronize()
            for j in range(2):
                suffix[i][j][rows, :, ln.long() - 1] = y[:, j::H // Hkv]
            y = att[i].decode(y[:, :, None], *pre[i], *suffix[i], ln)[0][:, :, 0]
            if sync:
                torch.cuda.synchronize()
        x.copy_(y)
        return x

    a = start()
    want = [token(*a, True).clone() for _ in range(tokens)]
    b = start()
    token(*b, False)              # warm up, then put everything back
    for t, u in zip((*b[0], *b[1], *b[2:]), (lambda s: (*s[0], *s[1], *s[2:]))(start())):
        t.copy_(u)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x = token(*b, False)
    for t, u in zip((*b[0], *b[1], *b[2:]), (lambda s: (*s[0], *s[1], *s[2:]))(start())):
        t.copy_(u)
    for i in range(tokens):
        g.replay()
        assert torch.equal(x, want[i]), i
    assert all(torch.equal(p, q) for p, q in zip(a[0], b[0]))
    assert torch.isfinite(x.float()).all() and not torch.equal(want[0], want[1])
    assert all(p.read_status() == 0 for p in lin + att)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_largest_batch(sca, dtype):
    """65535 heads over the batch, three rows each, then a token; and as many
    heads behind a short prefix.  References in 64 bits."""
    B, H, S, D = 13107, 5, 3, 64
    q, k, v, do = (rnd(B, H, S, D, seed=i, dtype=dtype) for i in range(4))
    decay = torch.tensor([-0.01, -0.1, -0.3, -1.0, -3.0], device="cuda")
    lam = torch.exp(decay.double())[:, None, None]
    plan = sca.DecayLinearAttention(B, H, S, D, decay, dtype=dtype, backward=True)
    o, end = plan.forward(q, k, v)
    dq, dk, dv, _ = plan.backward(do)
    tc = dtype == torch.bfloat16
    half = 2.0 ** -8 if tc else 2.0 ** -24

    def near(got, ref, mag, rounds):
        # 2 D + 16 roundings of fp32 a term; bf16: P once, and the result
        bound = 1.01 * half * ref.abs() + ((2 * D + 16) * 2.0 ** -23 + rounds) * mag
        assert ((got.double() - ref).abs() <= bound).all()

    x = [t.double() for t in (q, k, v, do)]
    y = [t.abs() for t in x]
    r = 2.0 ** -8 if tc else 0.0
    for name in ("o", "dq", "dk", "dv"):
        a, b, c, rev = {"o": (0, 1, 2, 0), "dq": (3, 2, 1, 0), "dk": (2, 3, 0, 1), "dv": (1, 0, 3, 1)}[name]
        w = torch.zeros(H, S, S, dtype=torch.float64, device="cuda")
        for i in range(S):
            for j in range(S):
                if (j >= i if rev else j <= i):
                    w[:, i, j] = torch.exp(decay.double() * abs(i - j))
        sums = [plan.scale * (w * (z[a] @ z[b].transpose(-1, -2))) @ z[c] for z in (x, y)]
        near({"o": o, "dq": dq, "dk": dk, "dv": dv}[name], *sums, r)
    state = torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda")
    for t in range(S):
        state = lam * state + x[1][:, :, t, :, None] * x[2][:, :, t, None, :]
    # sums of three terms, kept to 2^-16 or better where weights are below 1/16 (2^-20 of it)
    mag = sum(lam ** (S - 1 - t) * y[1][:, :, t, :, None] * y[2][:, :, t, None, :] for t in range(S))
    assert ((end.double() - state).abs() <= (20 * 2.0 ** -23) * mag).all()
    one = [t[:, :, 0] for t in (q, k, v)]
    mag = lam * mag + y[1][:, :, 0, :, None] * y[2][:, :, 0, None, :]
    got = plan.step(*one, end)
    state = lam * state + x[1][:, :, 0, :, None] * x[2][:, :, 0, None, :]
    ref, m = (plan.scale * (z[0][:, :, :1] @ st)[:, :, 0] for z, st in ((x, state), (y, mag)))
    near(got, ref, m, 0.0)
    del state, mag, x, y, sums
    n, cap = 100, 4
    qd = rnd(B, H, 1, D, seed=11, dtype=dtype)
    kp, vp = (rnd(H, n, D, seed=12 + i, dtype=dtype) for i in range(2))
    ks, vs = (rnd(B, H, cap, D, seed=14 + i, dtype=dtype) for i in range(2))
    ln = torch.arange(B, dtype=torch.int32, device="cuda") % (cap + 1)
    dec = sca.SharedPrefixAttention(B, H, D, n, cap, dtype=dtype)
    od, lse = dec.decode(qd, kp, vp, ks, vs, ln)
    qq = qd.double()
    s = dec.scale * torch.cat((torch.einsum("bhtd,hnd->bhtn", qq, kp.double()),
                               torch.einsum("bhtd,bhnd->bhtn", qq, ks.double())), -1)
    s = s.masked_fill((torch.arange(n + cap, device="cuda") >= n + ln[:, None])[:, None, None], -math.inf)
    p = s.softmax(-1)
    ref, m = (torch.einsum("bhtn,hnd->bhtd", p[..., :n], f(vp.double())) +
              torch.einsum("bhtn,bhnd->bhtd", p[..., n:], f(vs.double())) for f in (lambda t: t, torch.abs))
    # a weight errs by its score's error, (D + 2) 2^-23 |q||k| scale < 1e-4 here, and the sums' 104 roundings
    assert ((od.double() - ref).abs() <= 1.01 * half * ref.abs() + (3e-4 + r) * m).all()
    assert ((lse.double() - s.logsumexp(-1)).abs() <= 3e-4).all()
    assert plan.read_status() == 0 and dec.read_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("prefix,cap", [(0, 0), (50, 40)])
def test_nothing_to_attend_to(sca, dtype, prefix, cap):
    """No keys at all, caches left out, suffixes of length zero, caches of no rows."""
    B, H, Hkv, T, D = 3, 4, 2, 2, 64
    plan = sca.SharedPrefixAttention(B, H, D, prefix, cap, kv_heads=Hkv, tokens=T, dtype=dtype)
    q, none = rnd(B, H, T, D, dtype=dtype), rnd(Hkv, 0, D, dtype=dtype)
    ln = torch.zeros(B, dtype=torch.int32, device="cuda")
    calls = [(None, None, None, None, None), (none, none, None, None, ln)]
    if cap:
        s = rnd(B, Hkv, cap, D, seed=1, dtype=dtype)
        calls += [(None, None, s, s, ln), (none, none, s, s, ln)]
    for args in calls:
        plan.o.fill_(7)
        plan.lse.fill_(7)
        o, lse = plan.decode(q, *args)
        assert not o.any() and torch.isneginf(lse).all()
    assert plan.read_status() == 0
