"""GPU parity of linear attention with a decay per head (prompts, gradients,
single tokens) against the fp64 recurrence.

Bounds, element by element, from the roundings that the kernels make.  Let A
be the same sums over the inputs' magnitudes, and c the number of roundings
that one term of a result can pass through in sequence: D for the inner
product, D and a chunk's rows for the two sums, two per chunk for the carried
state, 16 for the weights.  fp32 arithmetic then errs by at most c 2^-24 A.
The tensor cores' accumulation may truncate instead of rounding (a step
instead of half of one: c 2^-23 A), and the kernels round the masked product
and the queries' copy of the state to bf16: half a step each of the terms
they are part of, 2^-8 A together, since every term is in one of the two.  A
bf16 result adds half a step of itself.  (A itself is computed from magnitudes, so it
bounds the value that each rounding is relative to.)  In the 2-norm the three
bf16 roundings are independent and spread evenly over their step (rms 2^-8 /
sqrt 3 of a value at most): sqrt(3) of that is 2^-8 of the norm.  States stay
fp32 throughout: roundings of random sign add up to sqrt(c) 2^-23 of the norm."""
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


def make(B, H, S, D, dtype, seed, lengths=None, poison=True):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(B, H, S, D, generator=g).to(dtype) for _ in range(4)]
    s0, ds = (torch.randn(B, H, D, D, generator=g) for _ in range(2))
    decay = -torch.exp(torch.linspace(math.log(1.5), math.log(2e-3), H)) if H > 1 else torch.tensor([-0.01])
    if lengths is not None and poison:
        for b, n in enumerate(lengths):
            for t in x:
                t[b, :, max(0, n):] = float("nan")
    return x, s0, ds, decay


def steps(S, D, chunk=64):
    return 2 * D + chunk * 2 + 2 * (S // chunk + 1) + 16


def close(name, got, ref, mag, dtype, c, tc):
    g, ref, mag = got.double().cpu().numpy(), np.asarray(ref), np.asarray(mag)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{name}: non-finite values"
    bound = HALF[dtype] * np.abs(ref) * 1.01 + (c * 2.0 ** -23 + (2.0 ** -8 if tc else 0.0)) * mag + 1e-37
    bad = np.abs(g - ref) > bound
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} beyond the bound, worst "
                           f"{(np.abs(g - ref) / bound).max():.2f} of it at {np.argwhere(bad)[0]}")
    norm = np.linalg.norm(ref)
    if norm:
        off = np.linalg.norm(g - ref) / norm
        most = 2.0 ** -8 if dtype == torch.bfloat16 else math.sqrt(c) * 2.0 ** -23
        assert off <= most, f"{name}: {off:.3e} of the norm, at most {most:.3e}"


def magnitudes(x, decay, scale, s0, ds, lengths):
    a = [torch.nan_to_num(t.double(), nan=0.0).abs() for t in x]
    s = abs(scale)
    s0, ds = (None if t is None else t.abs() for t in (s0, ds))
    fwd = oracle.decay_attention(*a[:3], decay, s, s0, lengths)
    return fwd + oracle.decay_attention_backward(*a, decay, s, s0, ds, lengths)


CASES = [
    # B, H, S, D, dtype, lengths, state
    (1, 1, 1, 64, "bf16", None, False), (2, 3, 2, 128, "bf16", None, True), (1, 2, 63, 128, "f32", None, True),
    (2, 2, 64, 64, "f32", [64, 1], False), (1, 2, 65, 64, "bf16", None, True), (2, 1, 127, 128, "bf16", [127, 0], True),
    (1, 2, 128, 128, "bf16", None, False), (3, 2, 129, 128, "bf16", [128, 129, 1], True),
    (1, 3, 255, 64, "bf16", None, True), (2, 2, 300, 128, "f32", [300, 130], True),
    (1, 4, 1025, 128, "bf16", None, True), (3, 2, 700, 64, "bf16", [700, 256, 257], True),
    (2, 2, 1000, 128, "bf16", [384, 1000], False), (1, 1, 2500, 64, "f32", None, True),
    (1, 2, 3300, 128, "bf16", [3000], True),
    (160, 2, 130, 64, "bf16", None, False),   # one segment each, more CTAs than SMs
]


@pytest.mark.parametrize("algo", ["auto", "simt"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:5]) + ("-ragged" if c[5] else ""))
def test_forward_and_backward_against_the_recurrence(sca, case, algo):
    B, H, S, D, dt, lengths, state = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    x, s0, ds, decay = make(B, H, S, D, dtype, seed=S + D, lengths=lengths)
    if not state:
        s0 = ds = None
    scale = 1 / math.sqrt(D)
    tc = algo == "auto" and dt == "bf16"
    plan = sca.DecayLinearAttention(B, H, S, D, decay, dtype=dtype, backward=True,
                                    algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    q, k, v, do = (t.cuda() for t in x)
    dev = lambda t: None if t is None else t.cuda()
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    # what is in the outputs from before must not show
    for t in (plan._o, plan._dq, plan._dk, plan._dv, plan.state, plan.dstate, plan._ws):
        t.fill_(float("nan"))
    o, end = plan.forward(q, k, v, state=dev(s0), lengths=ln)
    dq, dk, dv, first = plan.backward(do, dstate=dev(ds))
    assert plan.read_status() == 0
    ref = oracle.decay_attention(*x[:3], decay, scale, s0, lengths)
    ref += oracle.decay_attention_backward(*x, decay, scale, s0, ds, lengths)
    mag = magnitudes(x, decay, scale, s0, ds, lengths)
    c = steps(S, D)
    for name, got, r, m in zip(("o", "state", "dq", "dk", "dv", "dstate"), (o, end, dq, dk, dv, first), ref, mag):
        st = "state" in name
        if name == "dstate" and not state:
            assert got is None
            continue
        close(name, got, r, m, torch.float32 if st else dtype, c, tc and not st)
    if lengths is not None:
        for b, n in enumerate(lengths):
            for t in (o, dq, dk, dv):
                assert not t[b, :, n:].any(), "rows behind a sequence are zero"


@pytest.mark.parametrize("algo", ["auto", "simt"])
@pytest.mark.parametrize("g", [0.0, -1e-4, -3.0, -60.0, -1e30, -math.inf])
def test_decays_from_none_to_zero(sca, g, algo):
    B, H, S, D = 1, 2, 400, 128
    x, s0, ds, _ = make(B, H, S, D, torch.bfloat16, seed=9)
    decay = torch.tensor([g, -0.05])
    plan = sca.DecayLinearAttention(B, H, S, D, decay, backward=True,
                                    algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    q, k, v, do = (t.cuda() for t in x)
    o, end = plan.forward(q, k, v, state=s0.cuda())
    out = (o, end) + tuple(plan.backward(do, dstate=ds.cuda()))
    scale = 1 / math.sqrt(D)
    ref = oracle.decay_attention(*x[:3], decay, scale, s0)
    ref += oracle.decay_attention_backward(*x, decay, scale, s0, ds)
    mag = magnitudes(x, decay, scale, s0, ds, None)
    for name, got, r, m in zip(("o", "state", "dq", "dk", "dv", "dstate"), out, ref, mag):
        st = "state" in name
        close(name, got, r, m, torch.float32 if st else torch.bfloat16, steps(S, D), algo == "auto" and not st)


def test_gradients_against_differences(sca):
    """Central differences of <o, do> + <state, dstate> along a direction:
    the loss is linear in each input by itself, so in exact arithmetic the
    quotient has no truncation error.  What is left is fp32 rounding: each
    side of the difference errs by at most c 2^-23 times the loss's sum of
    magnitudes."""
    B, H, S, D = 1, 2, 333, 64
    x, s0, ds, decay = make(B, H, S, D, torch.float32, seed=3)
    plan = sca.DecayLinearAttention(B, H, S, D, decay, dtype=torch.float32, backward=True)
    q, k, v, do = (t.cuda() for t in x)
    s0, ds = s0.cuda(), ds.cuda()
    plan.forward(q, k, v, state=s0)
    grads = [t.double().clone() for t in plan.backward(do, dstate=ds)]
    mag = magnitudes(x, decay, plan.scale, s0.cpu(), ds.cpu(), None)
    total = float((torch.tensor(mag[0]) * x[3].double().abs()).sum() + (torch.tensor(mag[1]) * ds.cpu().double().abs()).sum())

    def loss(a):
        o, end = plan.forward(*a[:3], state=a[3])
        return float((o.double() * do.double()).sum() + (end.double() * ds.double()).sum())

    base = [q, k, v, s0]
    for i, name in enumerate(("q", "k", "v", "state")):
        d = torch.sign(grads[i]).float()      # the steepest direction: the quotient is the gradient's 1-norm
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + d, base[i] - d
        got = (loss(up) - loss(down)) / 2
        want = float((grads[i] * d.double()).sum())
        # the shifted inputs' magnitudes are at most three times as large (|x| + 1 against E|x| = 0.8)
        assert abs(got - want) <= 3 * steps(S, D) * 2.0 ** -23 * total, (name, got, want)
        assert abs(got - want) <= 1e-3 * abs(want), (name, got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views_of_a_fused_projection_and_a_shared_first_state(sca, dtype):
    B, H, S, D = 3, 4, 200, 64
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(B, S, 3, H, D, generator=g).to(dtype)
    s0 = torch.randn(1, H, D, D, generator=g)
    decay = torch.linspace(-0.5, -0.01, H)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    plan = sca.DecayLinearAttention(B, H, S, D, decay, dtype=dtype, backward=True)
    dev = qkv.cuda()
    o, end = plan.forward(*(dev[:, :, i].transpose(1, 2) for i in range(3)), state=s0.cuda().expand(B, H, D, D))
    ref = oracle.decay_attention(q, k, v, decay, plan.scale, s0)
    mag = oracle.decay_attention(q.abs(), k.abs(), v.abs(), decay, plan.scale, s0.abs())
    tc = dtype == torch.bfloat16
    close("o", o, ref[0], mag[0], dtype, steps(S, D), tc)
    close("state", end, ref[1], mag[1], torch.float32, steps(S, D), False)
    # do as a view as well; every sequence has its own gradient of the shared state
    do = torch.randn(B, S, H, D, generator=g).to(dtype)
    out = plan.backward(do.cuda().transpose(1, 2))
    ref = oracle.decay_attention_backward(q, k, v, do.transpose(1, 2), decay, plan.scale, s0)
    mag = oracle.decay_attention_backward(q.abs(), k.abs(), v.abs(), do.transpose(1, 2).abs(), decay, plan.scale, s0.abs())
    for name, got, r, m in zip(("dq", "dk", "dv", "dstate"), out, ref, mag):
        close(name, got, r, m, torch.float32 if name == "dstate" else dtype, steps(S, D), tc and name != "dstate")


def test_calls_of_fewer_rows_and_repeats_are_the_same_bits(sca):
    B, H, D = 2, 2, 128
    decay = torch.tensor([-0.2, -0.01])
    plan = sca.DecayLinearAttention(B, H, 1500, D, decay, backward=True)
    for S in (1500, 40, 700, 1, 1500):
        x, s0, ds, _ = make(B, H, S, D, torch.bfloat16, seed=S)
        q, k, v, do = (t.cuda() for t in x)
        outs = []
        for _ in range(2):
            o, end = plan.forward(q, k, v, state=s0.cuda())
            outs.append([t.clone() for t in (o, end, *plan.backward(do, dstate=ds.cuda()))])
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        alone = sca.DecayLinearAttention(B, H, S, D, decay, backward=True)
        o, end = alone.forward(q, k, v, state=s0.cuda())
        assert torch.equal(o, outs[0][0]) and torch.equal(end, outs[0][1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,D", [(1, 1, 64), (3, 5, 128), (2, 3, 64), (40, 16, 128), (330, 1, 64)])
def test_step(sca, B, H, D, dtype):
    g = torch.Generator().manual_seed(B + D)
    wide = torch.randn(B, 3, H, D, generator=g).to(dtype)      # a fused projection's output
    s0 = torch.randn(B, H, D, D, generator=g)
    decay = -torch.rand(H, generator=g)
    decay[0] = 0.0
    plan = sca.DecayLinearAttention(B, H, 1, D, decay, dtype=dtype)
    state, dev = s0.cuda(), wide.cuda()
    s = s0.double()
    a = s0.double().abs()
    for _ in range(3):
        o = plan.step(dev[:, 0], dev[:, 1], dev[:, 2], state)
        lam = torch.exp(decay.double())[:, None, None]
        q, k, v = (wide[:, i].double() for i in range(3))
        s = lam * s + k[..., None] * v[..., None, :]
        a = lam * a + (k[..., None] * v[..., None, :]).abs()
        ref = plan.scale * torch.einsum("bhd,bhde->bhe", q, s)
        mag = plan.scale * torch.einsum("bhd,bhde->bhe", q.abs(), a)
        # fp32: two roundings and the weight's a step, then a sum of D terms
        close("o", o, ref.numpy(), mag.numpy(), dtype, D + 20, False)
        close("state", state, s.numpy(), a.numpy(), torch.float32, 20, False)


@pytest.mark.parametrize("lengths", [None, [300, 10]])
def test_a_prompt_in_shards_and_single_tokens_is_the_prompt(sca, lengths):
    """Used together: a prompt in two shards that hand the state on, then
    single tokens, against the whole sequence at once.  Ragged prompts go on
    from their own last rows."""
    B, H, S, D, n_new = 2, 4, 300, 128, 5
    x, _, _, decay = make(B, H, S + n_new, D, torch.bfloat16, seed=77)
    q, k, v = (t.cuda() for t in x[:3])
    ln = lengths or [S] * B
    half = 150
    plan = sca.DecayLinearAttention(B, H, half, D, decay)
    outs, state = [], None
    for r in range(2):
        rows = slice(r * half, (r + 1) * half)
        part = torch.tensor([min(max(n - r * half, 0), half) for n in ln], dtype=torch.int32, device="cuda")
        o, state = plan.forward(q[:, :, rows], k[:, :, rows], v[:, :, rows], state=state, lengths=part)
        outs.append(o.clone())
    state = state.clone()
    at = torch.tensor(ln)
    new = [plan.step(*(torch.stack([t[b, :, at[b] + i] for b in range(B)]) for t in (q, k, v)), state).clone()
           for i in range(n_new)]
    scale = plan.scale
    for b in range(B):
        n = ln[b] + n_new
        xs = [t[b:b + 1, :, :n] for t in x[:3]]
        ref = oracle.decay_attention(*xs, decay, scale)
        mag = oracle.decay_attention(*(t.abs() for t in xs), decay, scale)
        got = torch.cat([torch.cat(outs, 2)[b:b + 1, :, :ln[b]]] + [t[b:b + 1, :, None] for t in new], 2)
        close("o", got, ref[0], mag[0], torch.bfloat16, steps(S, D), True)
        close("state", state[b:b + 1], ref[1], mag[1], torch.float32, steps(S, D), False)


def test_captured_and_replayed(sca):
    B, H, S, D = 2, 4, 500, 128
    x, s0, ds, decay = make(B, H, S, D, torch.bfloat16, seed=5)
    q, k, v, do = (t.cuda() for t in x)
    s0, ds = s0.cuda(), ds.cuda()
    ln = torch.tensor([500, 222], dtype=torch.int32, device="cuda")
    plan = sca.DecayLinearAttention(B, H, S, D, decay, backward=True)

    def all_of_it():
        o, end = plan.forward(q, k, v, state=s0, lengths=ln)
        return (o, end, *plan.backward(do, dstate=ds))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_of_it()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_of_it()
    # the replay reads what is in the inputs and the lengths then
    q.copy_(torch.randn_like(q))
    ln.copy_(torch.tensor([1, 499], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    want = [t.clone() for t in all_of_it()]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert plan.read_status() == 0


def test_long_sequence_sampled(sca):
    """32K rows on few heads, cut into many segments: rows of the end against
    the recurrence from the state that the rows before them leave, which the
    fp32 kernels (held to the recurrence above) sum.  Decays below e^-0.05
    forget 2000 rows to e^-100."""
    B, H, S, D = 1, 16, 32768, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn(B, H, S, D, generator=g, device="cuda").bfloat16() for _ in range(4))
    decay = torch.linspace(-1.0, -0.05, H)
    plan = sca.DecayLinearAttention(B, H, S, D, decay, backward=True)
    o, end = plan.forward(q, k, v)
    dq, dk, dv, _ = plan.backward(do)
    assert plan.read_status() == 0
    for lo in (0, 3968, S - 2304):
        rows = slice(lo, lo + 2304)
        x = [t[:, :, rows].cpu() for t in (q, k, v, do)]
        ref = oracle.decay_attention(*x[:3], decay, plan.scale)
        ref += oracle.decay_attention_backward(*x, decay, plan.scale)
        mag = magnitudes(x, decay, plan.scale, None, None, None)
        # 2000 rows from the cut nothing of the other side is left
        o_rows = slice(0 if lo == 0 else 2000, 2304)
        k_rows = slice(0, 2304 if lo + 2304 == S else 304)
        for name, got, i, keep in (("o", o, 0, o_rows), ("dq", dq, 2, o_rows), ("dk", dk, 3, k_rows), ("dv", dv, 4, k_rows)):
            close(name, got[:, :, rows][:, :, keep], ref[i][:, :, keep], mag[i][:, :, keep], torch.bfloat16,
                  steps(S, D), True)
        if lo + 2304 == S:
            close("state", end, ref[1], mag[1], torch.float32, steps(2304, D), False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S", [100, 3000])
def test_states_handed_back_in_place(sca, S, dtype):
    """A plan's own states as the next shard's, one segment and many: the same
    bits as from a copy."""
    B, H, D = 2, 2, 64
    x, s0, _, decay = make(B, H, S, D, dtype, seed=S)
    q, k, v = (t.cuda() for t in x[:3])
    ln = torch.tensor([S, 0], dtype=torch.int32, device="cuda")
    a, b = (sca.DecayLinearAttention(B, H, S, D, decay, dtype=dtype) for _ in range(2))
    a.forward(q, k, v, state=s0.cuda())
    b.forward(q, k, v, state=s0.cuda())
    for lengths in (None, ln):
        o, end = a.forward(q, k, v, state=a.state, lengths=lengths)
        o2, end2 = b.forward(q, k, v, state=b.state.clone(), lengths=lengths)
        assert torch.equal(o, o2) and torch.equal(end, end2)
    assert torch.equal(end[1], end2[1]) and not o[1].any()
