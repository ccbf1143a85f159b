"""GPU parity of rotary positions against the fp64 oracle, whose angles are
reduced in exact arithmetic.

Bounds.  What is left of an angle after the quarters is at most pi / 4 and is
rounded once (2^-24 of it: 0.79 2^-24), after 2^-32 turns were cut off
(0.025 2^-24); sincospi is within one unit (2^-24 of numbers below one); the
amplitude is rounded to fp32 and multiplied in (2^-24 each): each coefficient is
off by at most m E, E = 4 2^-24.  The result adds the two products' roundings,
2^-24 (|x_b s| + |y|).  So |error| <= m (|x_a| + |x_b|) 6 2^-24, plus half a step
of a bf16 output."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sca():
    import sharded_causal_softmax_gb300 as m
    from sharded_causal_softmax_gb300 import build
    build.build()
    return m


def rnd(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def check(y, x, cos, sin, angles, transposed=False):
    ref = oracle.rotary(x, cos, sin, angles.layout, angles.amplitude, transposed)
    pairs = oracle.rotary(x.double().abs(), np.ones_like(cos), np.ones_like(sin), angles.layout, angles.amplitude,
                          True)   # m (|x_a| + |x_b|) in the first place of every pair
    n, got = cos.shape[-1], y.double().cpu().numpy()
    i = np.arange(n)
    a, b = (i, i + n) if angles.layout == "half" else (2 * i, 2 * i + 1)
    mag = np.zeros_like(got)
    mag[..., a] = mag[..., b] = np.abs(pairs[..., a])
    bound = mag * 6 * 2.0 ** -24 + HALF[y.dtype] * 1.01 * np.abs(ref)
    # bf16 below the smallest normal number has steps of its own
    assert (np.abs(got - ref) <= bound + 1e-38).all(), (np.abs(got - ref) / np.maximum(bound, 1e-38)).max()
    assert torch.equal(y[..., angles.rotary_dim:].cpu(), x[..., angles.rotary_dim:])


CASES = [
    # B, H, Hkv, S, D, rotary_dim, layout, scaling, dtype, positions
    (1, 1, 1, 1, 64, 64, "half", None, "bf16", None), (2, 3, 1, 7, 128, 128, "half", None, "bf16", "given"),
    (3, 4, 2, 33, 64, 32, "interleaved", ("linear", 4.0), "f32", "shared"),
    (2, 9, 3, 129, 128, 64, "interleaved", ("ramp", 8.0, 4096), "bf16", "given"),
    (1, 12, 12, 500, 64, 64, "half", ("base", 4.0), "f32", None),
    (2, 2, 2, 65, 80, 48, "half", None, "bf16", "given"), (1, 5, 1, 40, 256, 96, "interleaved", None, "f32", None),
    # sizes that vectors of 16 bytes do not divide
    (2, 3, 2, 19, 40, 20, "half", None, "bf16", "given"), (1, 2, 1, 30, 66, 66, "interleaved", None, "bf16", None),
    (2, 2, 2, 11, 34, 2, "half", ("base", 2.0), "f32", "given"), (1, 1, 3, 5, 2, 2, "interleaved", None, "f32", None),
    (2, 33, 7, 70, 64, 64, "half", ("ramp", 4.0, 2048, 2.0, 8.0), "bf16", "shared"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_against_the_oracle(sca, case):
    B, H, Hkv, S, D, rd, layout, scaling, dt, given = case
    dtype = DT[dt]
    angles = sca.RotaryAngles(rd, layout=layout, scaling=scaling)
    q, k, dq, dk = (rnd(B, h, S, D, seed=i, dtype=dtype) for i, h in enumerate((H, Hkv, H, Hkv)))
    pos = torch.arange(S, dtype=torch.int32)
    if given:
        shape = (S,) if given == "shared" else (B, S)
        pos = torch.randint(0, 100000, shape, generator=torch.Generator().manual_seed(9), dtype=torch.int32)
    cos, sin = oracle.rotary_cos_sin(pos.expand(B, S).numpy(), angles.frequencies)
    cos, sin = cos[:, None], sin[:, None]
    plan = sca.RotaryPositions(B, H, S, D, angles, kv_heads=Hkv, dtype=dtype, backward=True)
    plan._own.fill_(float("nan"))
    dev = pos.cuda() if given else None
    q1, k1 = plan.forward(q.cuda(), k.cuda(), positions=dev)
    check(q1, q, cos, sin, angles)
    check(k1, k, cos, sin, angles)
    g1, g2 = plan.backward(dq.cuda(), dk.cuda())
    check(g1, dq, cos, sin, angles, transposed=True)
    check(g2, dk, cos, sin, angles, transposed=True)
    # a difference along any direction is the rotation of that direction: <y', R x> = <R^T y', x>
    if dt == "f32":
        lhs = (q1.double() * dq.cuda().double()).sum().item()
        rhs = (q.cuda().double() * g1.double()).sum().item()
        size = (q.double().norm() * dq.double().norm()).item() * angles.amplitude
        assert abs(lhs - rhs) <= 2 * 6 * 2.0 ** -24 * 2 * size


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_positions_at_the_ends_of_their_range(sca, layout):
    """Far positions lose nothing: the bound is that of near ones."""
    rd = D = 64
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, 1234567891, -987654321], dtype=torch.int32)
    x = rnd(1, 2, len(pos), D, seed=3, dtype=torch.float32)
    for freq in (None, [0.0, 1e-12, 2.5, 100.0, 3.0e9, -1.0] + [float(i) for i in range(26)]):
        angles = sca.RotaryAngles(rd, layout=layout, frequencies=freq)
        cos, sin = oracle.rotary_cos_sin(pos.numpy(), angles.frequencies)
        plan = sca.RotaryPositions(1, 2, len(pos), D, angles, dtype=torch.float32)
        y, _ = plan.forward(x.cuda(), x.cuda(), positions=pos.cuda())
        check(y, x, cos, sin, angles)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_views(sca, dt):
    """Heads out of one projection's output, rows first; one key head for all
    requests; an address off a vector; fewer rows than the plan's."""
    B, H, Hkv, S, D = 3, 4, 2, 21, 64
    dtype = DT[dt]
    angles = sca.RotaryAngles(32, layout="interleaved")
    wide = rnd(B, S, H + 2 * Hkv, D, seed=1, dtype=dtype)
    one = rnd(1, Hkv, S, D, seed=2, dtype=dtype)
    plan = sca.RotaryPositions(B, H, 50, D, angles, kv_heads=Hkv, dtype=dtype)
    cos, sin = (x[None, None] for x in oracle.rotary_cos_sin(np.arange(S), angles.frequencies))
    dev, dev1 = wide.cuda(), one.cuda()
    q1, k1 = plan.forward(dev[:, :, :H].transpose(1, 2), dev1.expand(B, Hkv, S, D))
    check(q1, wide[:, :, :H].transpose(1, 2), cos, sin, angles)
    check(k1, one.expand(B, Hkv, S, D), cos, sin, angles)
    flat = torch.zeros(B * H * S * D + 1, dtype=dtype, device="cuda")
    off = flat[1:].view(B, H, S, D)
    off.copy_(dev[:, :, :H].transpose(1, 2))
    q2, _ = plan.forward(off, dev[:, :, H:H + Hkv].transpose(1, 2))
    check(q2, wide[:, :, :H].transpose(1, 2), cos, sin, angles)


def test_calls_that_are_refused(sca):
    angles = sca.RotaryAngles(64)
    plan = sca.RotaryPositions(2, 4, 16, 64, angles, kv_heads=2, backward=True)
    q, k = (rnd(2, h, 16, 64, seed=h, dtype=torch.bfloat16).cuda() for h in (4, 2))
    with pytest.raises(RuntimeError):
        plan.backward(q, k)
    q1, k1 = plan.forward(q, k)
    pos = torch.zeros(2, 16, dtype=torch.int32, device="cuda")
    for bad in ((q.float(), k), (q.cpu(), k), (q, q), (q[:, :, :8], k), (q.transpose(2, 3), k), (q1, k), (q, k1),
                (torch.cat([q, q], 2), torch.cat([k, k], 2)), (q[0], k[0])):
        with pytest.raises(ValueError):
            plan.forward(*bad)
    for bad in (pos.long(), pos.cpu(), pos[:1], pos[:, :8], torch.zeros(2, 32, dtype=torch.int32, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            plan.forward(q, k, positions=bad)
    plan.forward(q, k)
    with pytest.raises(ValueError):
        plan.backward(q[:, :, :8], k[:, :, :8])
    no = sca.RotaryPositions(2, 4, 16, 64, angles, kv_heads=2)
    no.forward(q, k)
    with pytest.raises(RuntimeError):
        no.backward(q, k)


def test_in_place_and_captured(sca):
    """The C function over its own inputs; a captured pass whose positions
    change between replays, on a side stream."""
    import ctypes
    capi = sca.capi
    B, H, S, D = 2, 3, 37, 128
    angles = sca.RotaryAngles(128)
    x = rnd(B, H, S, D, seed=5, dtype=torch.float32)
    d = capi.sca_rotary_dims()
    d.B, d.H, d.Hkv, d.D, d.S, d.dtype, d.rotary_dim, d.amplitude = B, H, 0, D, S, capi.SCA_F32, D, 1.0
    d.q = d.qo = capi.view(H * S * D, S * D, D)
    y = x.cuda()
    capi.rotary_apply(d, y.data_ptr(), None, angles.turns.data_ptr(), None, y.data_ptr(), None,
                      torch.cuda.current_stream().cuda_stream)
    cos, sin = (t[None, None] for t in oracle.rotary_cos_sin(np.arange(S), angles.frequencies))
    check(y, x, cos, sin, angles)
    assert ctypes.sizeof(d) > 0
    plan = sca.RotaryPositions(B, H, S, D, angles, dtype=torch.float32)
    pos = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    dev = x.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.forward(dev, dev, positions=pos)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q1, k1 = plan.forward(dev, dev, positions=pos)
    for shift in (7, 70000):
        p = torch.arange(S, dtype=torch.int32).expand(B, S) + shift
        pos.copy_(p)
        graph.replay()
        torch.cuda.synchronize()
        cos, sin = (t[:, None] for t in oracle.rotary_cos_sin(p.numpy(), angles.frequencies))
        check(q1, x, cos, sin, angles)
        assert torch.equal(q1, k1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_numbers_that_are_not_finite_stay_in_their_pair(sca, dt):
    B, H, S, D = 1, 2, 9, 64
    angles = sca.RotaryAngles(32, layout="half")
    x = rnd(B, H, S, D, seed=1, dtype=DT[dt]).cuda()
    plan = sca.RotaryPositions(B, H, S, D, angles, dtype=DT[dt])
    clean = plan.forward(x, x)[0].clone()
    x[0, 1, 4, 3] = float("nan")
    x[0, 0, 2, 40] = float("inf")   # behind the turned features: copied
    y = plan.forward(x, x)[0]
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 1, 4, 3] = want[0, 1, 4, 19] = want[0, 0, 2, 40] = True
    assert torch.equal(bad, want) and torch.equal(y[~want], clean[~want])


@pytest.mark.parametrize("schedule,layout,S,P", [("ring", "zigzag", 512, 2), ("fused", "contiguous", 384, 1),
                                                 ("direct", "zigzag", 120, 2)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_sharded_attention_turns_its_queries_and_keys(sca, schedule, layout, S, P, dt):
    """The plan with angles is the plan without, between a rotation before and
    the transposed one behind, bit for bit (the same kernels)."""
    B, H, Hkv, D = 2, 4, 2, 64
    dtype = DT[dt]
    angles = sca.RotaryAngles(32, scaling=("ramp", 4.0, 64))
    q, k, v, do = (rnd(B, h, S, D, seed=i, dtype=dtype).cuda() for i, h in enumerate((H, Hkv, Hkv, H)))
    pos = (torch.arange(S, dtype=torch.int32) * 3 + 11).cuda()
    make = lambda **kw: sca.ShardedCausalAttention(B, H, S, D, P, layout=layout, schedule=schedule, dtype=dtype,
                                                   kv_heads=Hkv, backward=True, **kw)
    whole, plain = make(rotary=angles), make()
    o, lse = (t.clone() for t in whole.forward(q, k, v, positions=pos))
    grads = [t.clone() for t in whole.backward(do)]
    again = [t.clone() for t in whole.backward(do, q, k, v)]
    assert whole.launches > 0 and whole.read_status() == 0
    before = sca.RotaryPositions(B, H, S, D, angles, kv_heads=Hkv, dtype=dtype)
    behind = sca.RotaryPositions(B, H, S, D, angles, kv_heads=Hkv, dtype=torch.float32, backward=True)
    q1, k1 = before.forward(q, k, positions=pos)
    o2, lse2 = plain.forward(q1, k1, v)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    dq, dk, dv = plain.backward(do)
    behind.forward(q.float(), k.float(), positions=pos)
    dq, dk = behind.backward(dq, dk)
    # dq is summed by atomics in no fixed order on the tensor cores: two runs differ by rounding
    for got in (grads, again):
        assert torch.equal(got[2], dv) and torch.equal(got[1], dk)
        assert (got[0] - dq).abs().max().item() <= 1e-5 * max(1.0, dq.abs().max().item())
    with pytest.raises(ValueError):
        plain.forward(q, k, v, positions=pos)
    with pytest.raises(ValueError):
        whole.forward(q, k, v, positions=pos[:5])


@pytest.mark.parametrize("kw", [dict(schedule="ring", addressing="permuted"), dict(schedule="ring", head_groups=2),
                                dict(schedule="direct", bf16_out=True), dict(schedule="ring", visit="double_ring", inner=2)],
                         ids=lambda kw: "-".join(str(x) for x in kw.values()))
def test_other_ways_to_shard_turn_them_alike(sca, kw):
    B, H, S, D, P = 1, 4, 1024, 128, 4 if "inner" in kw else 2
    angles = sca.RotaryAngles(128)
    q, k, v, do = (rnd(B, H, S, D, seed=20 + i, dtype=torch.bfloat16).cuda() for i in range(4))
    make = lambda **more: sca.ShardedCausalAttention(B, H, S, D, P, backward=True, **kw, **more)
    whole, plain = make(rotary=angles), make()
    o, lse = (t.clone() for t in whole.forward(q, k, v))
    grads = [t.clone() for t in whole.backward(do)]
    before = sca.RotaryPositions(B, H, S, D, angles)
    behind = sca.RotaryPositions(B, H, S, D, angles, dtype=torch.float32, backward=True)
    o2, lse2 = plain.forward(*before.forward(q, k), v)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    dq, dk, dv = (t.float() for t in plain.backward(do))
    behind.forward(q.float(), k.float())
    dq, dk = behind.backward(dq, dk)
    for got, want in zip(grads, (dq, dk, dv)):   # sums by atomics differ by rounding
        assert (got - want).abs().max().item() <= 1e-5 * max(1.0, want.abs().max().item())
    assert whole.read_status() == 0


def test_gradient_through_rotated_attention_against_differences(sca):
    """fp32: the loss sum(o * do) moved by small steps of q and k."""
    B, H, S, D = 1, 2, 64, 64
    angles = sca.RotaryAngles(64, layout="interleaved")
    q, k, v, do = (rnd(B, H, S, D, seed=10 + i, dtype=torch.float32) for i in range(4))
    plan = sca.ShardedCausalAttention(B, H, S, D, 1, layout="contiguous", dtype=torch.float32, backward=True,
                                      rotary=angles)
    plan.forward(q.cuda(), k.cuda(), v.cuda())
    dq, dk, _ = (t.double().cpu() for t in plan.backward(do.cuda()))
    cos, sin = (t[None, None] for t in oracle.rotary_cos_sin(np.arange(S), angles.frequencies))

    def loss(q, k):
        qq, kk = (oracle.rotary(t, cos, sin, "interleaved") for t in (q, k))
        o, _ = oracle.attention(qq, kk, v.double().numpy(), 1.0 / math.sqrt(D))
        return float((o * do.double().numpy()).sum())

    g = torch.Generator().manual_seed(0)
    for i, grad in ((0, dq), (1, dk)):
        for _ in range(3):
            step = torch.randn(B, H, S, D, generator=g, dtype=torch.float64)
            h = 1e-5
            x = [q.double(), k.double()]
            up, down = list(x), list(x)
            up[i], down[i] = x[i] + h * step, x[i] - h * step
            num = (loss(*(t.numpy() for t in up)) - loss(*(t.numpy() for t in down))) / (2 * h)
            ana = float((grad * step).sum())
            # fp32 gradients are off by 2e-4 an entry at most, independently along a random step; the
            # difference by h^2 times third derivatives and 1e-16 |loss| / h, both below 1e-7
            assert abs(num - ana) <= 2e-4 * float(step.norm())
