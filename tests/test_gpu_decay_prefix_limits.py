"""Decaying linear attention and shared-prefix decoding at the edges of what
the entry points take."""
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


def rnd(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


@pytest.mark.parametrize("dtype,algo", [(torch.bfloat16, "simt"), (torch.float32, "auto"), (torch.bfloat16, "auto")])
def test_more_query_rows_than_a_grid_axis_counts_blocks_of(sca, dtype, algo):
    """B R = 2162655 rows of the prefix: 67584 blocks of 32, an axis but the first holds 65535.

    Bounds: a score is off by D 2^-23 |q| |k| scale, the sums over n = 16 keys
    by n 2^-23, a bf16 weight by 2^-8, the output by half a step."""
    B, T, D, prefix, cap = 65535, 33, 64, 5, 11
    q = rnd(B, 1, T, D, seed=1, dtype=dtype)
    kp, vp = (rnd(1, prefix, D, seed=i, dtype=dtype) for i in (2, 3))
    ks, vs = (rnd(B, 1, cap, D, seed=i, dtype=dtype) for i in (4, 5))
    ln = (torch.arange(B, device="cuda") * 7 % (cap + 1)).int()
    plan = sca.SharedPrefixAttention(B, 1, D, prefix, cap, tokens=T, dtype=dtype,
                                     algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    plan.o.fill_(float("nan"))
    plan.lse.fill_(float("nan"))
    plan._ws.fill_(float("nan"))
    o, lse = plan.decode(q, kp, vp, ks, vs, ln)
    assert plan.read_status() == 0
    last = ln.long()[:, None] - (T - 1 - torch.arange(T, device="cuda"))                # [B, T]
    for b0 in range(0, B, 8192):                                                        # in 64 bits, a part at a time
        part = slice(b0, b0 + 8192)
        x, n = q[part, 0].double(), last[part]
        s = torch.cat([x @ kp[0].double().T, x @ ks[part, 0].double().transpose(1, 2)], 2) * plan.scale
        s[:, :, prefix:].masked_fill_(torch.arange(cap, device="cuda") >= n[..., None], -math.inf)
        p = torch.softmax(s, 2)
        vo = vs[part, 0].double()
        ref = p[..., :prefix] @ vp[0].double() + p[..., prefix:] @ vo
        mag = p[..., :prefix] @ vp[0].double().abs() + p[..., prefix:] @ vo.abs()
        top = max(float(kp.double().norm(dim=-1).max()), float(ks[part].double().norm(dim=-1).max()))
        es = D * 2.0 ** -23 * float(x.norm(dim=-1).max()) * top * plan.scale + 2.0 ** -21
        err = 2 * es + (prefix + cap) * 2.0 ** -23 + 2.0 ** -20
        if dtype == torch.bfloat16 and algo == "auto":
            err += 2.0 ** -8
        assert ((o[part, 0].double() - ref).abs() <= 1.01 * HALF[dtype] * ref.abs() + err * mag).all()
        rl = torch.logsumexp(s, 2)
        lb = es + (prefix + cap) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * rl.abs()
        assert ((lse[part, 0].double() - rl).abs() <= lb).all()


@pytest.mark.parametrize("dtype,algo", [(torch.bfloat16, "auto"), (torch.bfloat16, "simt"), (torch.float32, "auto")])
@pytest.mark.parametrize("S", [300, 2500])
@pytest.mark.parametrize("D", [64, 128])
def test_an_infinite_key_makes_infinities(sca, D, S, dtype, algo):
    """A key with an infinity in a live row (in a whole chunk, and in the
    ragged one at the end): its feature's row of the state becomes +-inf, the
    outputs from its row on follow, rows before it and other heads are what
    they were.  Decays of which the state takes two parts of the keys, and
    three, for all rows but the last."""
    H, decay = 2, [-0.04, -0.002]
    at = [(150, 5, math.inf), (S - 10, 7, -math.inf)]
    q, k, v = (rnd(1, H, S, D, seed=i, dtype=dtype) for i in range(3))
    plan = sca.DecayLinearAttention(1, H, S, D, decay, dtype=dtype,
                                    algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    for h in range(H):
        clean = [t.clone() for t in plan.forward(q, k, v)]
        kk = k.clone()
        for t, f, x in at:
            kk[0, h, t, f] = x
        with np.errstate(invalid="ignore"):
            ro, rs = oracle.decay_attention(*(t.cpu() for t in (q, kk, v)), torch.tensor(decay), plan.scale)
        o, state = (t.double().cpu().numpy() for t in plan.forward(q, kk, v))
        co, cs = (t.double().cpu().numpy() for t in clean)
        assert plan.read_status() == 0
        # the state: the two rows infinite as defined, all others unchanged
        other = [f for f in range(D) if f not in (5, 7)]
        for f in (5, 7):
            assert np.isinf(rs[0, h, f]).all() and np.array_equal(state[0, h, f], rs[0, h, f])
        assert np.array_equal(state[0, h][other], cs[0, h][other]) and np.array_equal(state[0, 1 - h], cs[0, 1 - h])
        # outputs: the same before, infinite or (two infinities against each other) NaN as defined behind
        assert np.array_equal(o[0, h, :150], co[0, h, :150]) and np.array_equal(o[0, 1 - h], co[0, 1 - h])
        assert not np.isfinite(ro[0, h, 150:]).any()
        assert np.array_equal(o[0, h, 150:], ro[0, h, 150:], equal_nan=True)


@pytest.mark.parametrize("dtype,algo", [(torch.bfloat16, "auto"), (torch.bfloat16, "simt"), (torch.float32, "auto")])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_value_that_is_not_finite_stays_in_its_feature_and_chunk(sca, bad, dtype, algo):
    """Never lost, and nowhere but in its own feature: of the rows that see it,
    of the state, and of its own chunk's rows before it."""
    H, S, D, t, e = 2, 300, 64, 150, 9
    chunk = 128 if dtype == torch.bfloat16 and algo == "auto" else 64
    q, k, v = (rnd(1, H, S, D, seed=i, dtype=dtype) for i in range(3))
    plan = sca.DecayLinearAttention(1, H, S, D, [-0.04, -0.002], dtype=dtype,
                                    algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    co, cs = (x.clone() for x in plan.forward(q, k, v))
    v[0, 0, t, e] = bad
    o, state = plan.forward(q, k, v)
    assert plan.read_status() == 0
    other = torch.arange(D, device="cuda") != e
    assert torch.equal(o[0, 1], co[0, 1]) and torch.equal(state[0, 1], cs[0, 1])
    assert torch.equal(o[0, 0][:, other], co[0, 0][:, other]) and torch.equal(state[0, 0][:, other], cs[0, 0][:, other])
    assert torch.equal(o[0, 0, :t // chunk * chunk, e], co[0, 0, :t // chunk * chunk, e])
    assert not torch.isfinite(o[0, 0, t:, e]).any() and not torch.isfinite(state[0, 0, :, e]).any()


@pytest.mark.parametrize("dtype,algo", [(torch.bfloat16, "auto"), (torch.bfloat16, "simt"), (torch.float32, "auto")])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_newest_tokens_value_that_is_not_finite_stays_in_its_feature(sca, bad, dtype, algo):
    """The last of three tokens: in every row that sees it, and nowhere but in
    its own request, key/value head and feature; its key is seen by its own rows alone."""
    B, Hkv, group, T, D, n, cap, e = 3, 2, 2, 3, 64, 300, 200, 9
    q = rnd(B, Hkv * group, T, D, seed=1, dtype=dtype)
    kp, vp, ks, vs = (rnd(*s, D, seed=2 + i, dtype=dtype) for i, s in
                      enumerate(((Hkv, n), (Hkv, n), (B, Hkv, cap), (B, Hkv, cap))))
    lengths = [150, 129, 3]
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    plan = sca.SharedPrefixAttention(B, Hkv * group, D, n, cap, kv_heads=Hkv, tokens=T, dtype=dtype,
                                     algo=sca.capi.SCA_ALGO_AUTO if algo == "auto" else sca.capi.SCA_ALGO_SIMT)
    for b in range(B):
        co, cl = (x.clone() for x in plan.decode(q, kp, vp, ks, vs, ln))
        v, k = vs.clone(), ks.clone()
        v[b, 1, lengths[b] - 1, e] = bad
        o, lse = plan.decode(q, kp, vp, ks, v, ln)
        mine = torch.zeros_like(o, dtype=torch.bool)
        mine[b, group:, :, e] = True
        assert torch.equal(o[~mine], co[~mine]) and torch.equal(lse, cl)
        assert not torch.isfinite(o[b, group:, T - 1, e]).any()
        k[b, 1, lengths[b] - 1, e] = math.nan
        o, lse = plan.decode(q, kp, vp, k, vs, ln)
        hit = torch.zeros_like(lse, dtype=torch.bool)
        hit[b, group:, T - 1] = True
        assert torch.equal(o[~hit], co[~hit]) and torch.equal(lse[~hit], cl[~hit]) and torch.isnan(lse[hit]).all()
        assert torch.isnan(o[hit]).all()
    assert plan.read_status() == 0


def make_backward(sca, B, H, S, D, dtype, ragged, state):
    x = [rnd(B, H, S, D, seed=i, dtype=dtype) for i in range(4)]
    lengths = torch.tensor([S - (S // 3) * b for b in range(B)], dtype=torch.int32, device="cuda") if ragged else None
    s0, ds = (rnd(B, H, D, D, seed=i, dtype=torch.float32) if state else None for i in (7, 8))
    decay = [-0.5 / 10 ** h for h in range(H)]
    return sca.DecayLinearAttention(B, H, S, D, decay, dtype=dtype, backward=True), x, lengths, s0, ds


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("state", [False, True])
def test_backward_without_what_the_forward_left(sca, dtype, ragged, state):
    """ws_holds_forward = 0: the states before the segments are summed again,
    to the same bits, whatever the workspace held."""
    B, H, S, D = 2, 3, 3000, 64
    plan, x, lengths, s0, ds = make_backward(sca, B, H, S, D, dtype, ragged, state)
    assert plan._ws.numel() > 1   # cut into segments
    c_fwd = [t.clone() for t in plan.forward(*x[:3], state=s0, lengths=lengths)]
    want = [None if t is None else t.clone() for t in plan.backward(x[3], dstate=ds)]

    capi = sca.capi
    d = plan._make_dims(S, *((H * S * D, S * D, D),) * 3)
    ptr = lambda t: None if t is None else t.data_ptr()
    one = H * D * D
    stream = torch.cuda.current_stream().cuda_stream
    nan = lambda t: torch.full_like(t, float("nan"))
    o, end = nan(c_fwd[0]), nan(c_fwd[1])
    ws = nan(plan._ws)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = plan.log_decay
    capi.decay_attn_fwd(d, *map(ptr, x[:3]), ptr(g), ptr(lengths), ptr(s0), one, ptr(o), ptr(end), ptr(ws),
                        ws.numel() * 4, ptr(status), stream)
    assert torch.equal(o, c_fwd[0]) and torch.equal(end, c_fwd[1])
    got = [nan(t) for t in x[:3]] + [nan(end) if state else None]
    ws.fill_(float("nan"))
    capi.decay_attn_bwd(d, *map(ptr, x), capi.view(H * S * D, S * D, D), ptr(g), ptr(lengths), ptr(s0), one, ptr(ds),
                        one, *map(ptr, got), ptr(ws), ws.numel() * 4, 0, ptr(status), stream)
    assert capi.sca_read_status(ptr(status), stream) == 0
    for name, a, b in zip(("dq", "dk", "dv", "dstate"), got, want):
        assert (a is None and b is None) or torch.equal(a, b), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_step_and_decode_by_the_c_functions(sca, dtype):
    """The same bits as the plans' calls."""
    capi = sca.capi
    stream = torch.cuda.current_stream().cuda_stream
    B, H, D = 3, 4, 64
    lin = sca.DecayLinearAttention(B, H, 1, D, [-0.1] * H, dtype=dtype)
    x = [rnd(B, H, D, seed=i, dtype=dtype) for i in range(3)]
    a = rnd(B, H, D, D, seed=5, dtype=torch.float32)
    b = a.clone()
    want = lin.step(*x, a).clone()
    o = torch.full_like(want, float("nan"))
    capi.decay_attn_step(lin._make_dims(1, *((H * D, D, D),) * 3), *(t.data_ptr() for t in x),
                         lin.log_decay.data_ptr(), b.data_ptr(), H * D * D, o.data_ptr(), stream)
    assert torch.equal(o, want) and torch.equal(a, b)

    n, cap = 300, 70
    plan = sca.SharedPrefixAttention(B, H, D, n, cap, kv_heads=2, dtype=dtype)
    args = [rnd(B, H, 1, D, seed=1, dtype=dtype)] + [rnd(*s, D, seed=i, dtype=dtype) for i, s in
                                                   enumerate(((2, n), (2, n), (B, 2, cap), (B, 2, cap)))]
    ln = torch.tensor([70, 0, 33], dtype=torch.int32, device="cuda")
    want = [t.clone() for t in plan.decode(*args, ln)]
    o, lse, ws = (torch.full_like(t, float("nan")) for t in (plan.o, plan.lse, plan._ws))
    capi.prefix_attn_decode(plan._make_dims(H * D, n, cap, (n * D, D), (2 * cap * D, cap * D, D)),
                            *(t.data_ptr() for t in args), ln.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                            ws.numel() * 4, plan.status.data_ptr(), stream)
    assert plan.read_status() == 0 and torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_a_plans_states_are_refused_as_inputs(sca):
    """An fp32 plan's states have a shape that rows of inputs may have; written
    while they are read, they would give something else."""
    B, H, D = 2, 3, 64
    lin = sca.DecayLinearAttention(B, H, D, D, [-0.1] * H, dtype=torch.float32, backward=True)
    x = [rnd(B, H, D, D, seed=i, dtype=torch.float32) for i in range(4)]
    s0 = rnd(B, H, D, D, seed=9, dtype=torch.float32)
    lin.forward(*x[:3], state=s0)
    ds = lin.backward(x[3])[3]
    for t in (lin.state, ds):
        for i in range(3):
            args = list(x[:3])
            args[i] = t
            with pytest.raises(ValueError):
                lin.forward(*args)
            one = [y[:, :, 0] for y in x[:3]]
            one[i] = t[:, :, 5]
            with pytest.raises(ValueError):
                lin.step(*one, s0)
    for t in (lin.state, ds):
        lin.forward(*x[:3], state=s0)
        with pytest.raises(ValueError):
            lin.backward(t)
    odd = torch.zeros(B * H * D * D + 4, device="cuda")
    with pytest.raises(ValueError):
        lin.step(*(y[:, :, 0] for y in x[:3]), odd[1:1 + s0.numel()].view_as(s0))
    lin.step(*(y[:, :, 0] for y in x[:3]), lin.state)   # in place is what a step does
