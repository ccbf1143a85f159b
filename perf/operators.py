"""Cases for measuring two operators that serve and train long sequences, and
their plain forms.

Causal linear attention with a decay for each head.  With g_h <= 0 the log of
head h's decay and S_t a D x D state,

    S_t = exp(g_h) S_{t-1} + k_t^T v_t,      o_t = scale * q_t S_t,

is taken over whole prompts (``prompt``: outputs and the state after the last
row), over a training step (``train``: the same, and the gradients of q, k, v
and of the first state) and one token at a time (``step``: the state updated in
place).  Rows at or past a sequence's length give zeros and touch no state.

Attention of a decode step for a batch that shares a long prefix (``decode``):
every request's T newest tokens attend to the prefix's keys, kept once for the
whole batch, and to the request's own suffix cache, whose last T keys are the
tokens themselves: token t sees the suffix keys below length - (T - 1 - t).
Grouped-query heads; o and the natural-log lse of every query row.

Where ``own`` is false ``run`` computes them with elementary torch operations.
"""
import math
import random

import torch

own = False

CHUNK = 128   # rows of a chunk of the plain chunked form

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a chat turn's short prompt on a small model: latency
        dict(name="prompt_short", op="prompt", B=1, H=8, S=77, D=64, dtype="bf16", ragged=False, state=False),
        # a batch of prompts of mixed lengths, each going on from the state of a shared preamble
        dict(name="prompt_batch", op="prompt", B=8, H=16, S=2049, D=128, dtype="bf16", ragged=True, state=True),
        # one long document, few heads: the sequence itself has to fill the card
        dict(name="prompt_long", op="prompt", B=1, H=16, S=32768, D=128, dtype="bf16", ragged=False, state=False),
        # fine-tuning on short padded samples
        dict(name="train_padded", op="train", B=6, H=8, S=500, D=64, dtype="bf16", ragged=True, state=False),
        # a numerics run in full precision
        dict(name="train_f32", op="train", B=1, H=8, S=1000, D=64, dtype="f32", ragged=False, state=True),
        # the repository's linear-attention training step: 16 heads of 32K rows
        dict(name="train_32k", op="train", B=1, H=16, S=32768, D=128, dtype="bf16", ragged=False, state=False),
        # one request's next token: latency
        dict(name="step_one", op="step", B=1, H=16, D=128, dtype="bf16"),
        # a small batch of a model that keeps its activations in 32 bits
        dict(name="step_f32", op="step", B=33, H=12, D=64, dtype="f32"),
        # a full batch: the states stream through the card
        dict(name="step_batch", op="step", B=256, H=16, D=128, dtype="bf16"),
        # a few requests behind a short system prompt, every head its own keys: latency
        dict(name="decode_short", op="decode", B=4, Hkv=8, group=1, T=1, prefix=500, suffix=64, D=64, dtype="bf16"),
        # tokens proposed ahead and verified together, an odd group of heads
        dict(name="decode_verify", op="decode", B=13, Hkv=4, group=5, T=3, prefix=8191, suffix=700, D=128,
             dtype="bf16"),
        # a full batch behind a book-length prefix, the repository's 32 heads on 8 key/value heads
        dict(name="decode_long", op="decode", B=64, Hkv=8, group=4, T=1, prefix=131072, suffix=2048, D=128,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "train", "step", "decode"))
    D = rng.choice((64, 128))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op in ("prompt", "train"):
        cap = (1 << 26 if dtype == "bf16" else 1 << 23) // D
        B, H = _log_int(rng, 1, 16), _log_int(rng, 1, 32)
        S = _log_int(rng, 1, min(65536 if op == "prompt" else 32768, max(1, cap // (B * H))))
        return dict(op=op, B=B, H=H, S=S, D=D, dtype=dtype, ragged=rng.random() < 0.5, state=rng.random() < 0.5)
    if op == "step":
        B, H = _log_int(rng, 1, 256), _log_int(rng, 1, 32)
        return dict(op=op, B=max(1, min(B, 4096 // H)), H=H, D=D, dtype=dtype)
    Hkv, group, T = _log_int(rng, 1, 8), _log_int(rng, 1, 16), rng.choice((1, 1, 1, 2, 4))
    B = _log_int(rng, 1, 64)
    most = 2048 * 131072 if dtype == "bf16" else 1 << 22   # query rows x keys
    rows = B * Hkv * group * T
    prefix = _log_int(rng, 1, max(1, min(131072, most // rows)))
    suffix = _log_int(rng, T, max(T, min(2048, most // (8 * rows) + T)))
    return dict(op=op, B=B, Hkv=Hkv, group=group, T=T, prefix=prefix, suffix=suffix, D=D, dtype=dtype)


def _lengths(case):
    """Lengths of the sequences (prompt, train) or of the suffixes (decode): the case's own, the same for every seed."""
    B = case["B"]
    if case["op"] == "decode":
        rng = random.Random(7 * B + case["suffix"])
        return [rng.randint(min(case["T"], case["suffix"]), case["suffix"]) for _ in range(B)]
    if not case["ragged"]:
        return [case["S"]] * B
    rng = random.Random(11 * B + case["S"])
    return [case["S"]] + [rng.randint(max(1, case["S"] // 4), case["S"]) for _ in range(B - 1)]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[case["dtype"]]

    def rnd(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    st = {"case": case, "scale": 1.0 / math.sqrt(case["D"])}
    D = case["D"]
    if case["op"] == "decode":
        B, Hkv, T, H = case["B"], case["Hkv"], case["T"], case["Hkv"] * case["group"]
        st["q"] = rnd(B, H, T, D)
        st["kp"], st["vp"] = rnd(Hkv, case["prefix"], D), rnd(Hkv, case["prefix"], D)
        st["ks"], st["vs"] = rnd(B, Hkv, case["suffix"], D), rnd(B, Hkv, case["suffix"], D)
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
        if own:
            import sharded_causal_softmax_gb300 as sca
            st["plan"] = sca.SharedPrefixAttention(B, H, D, case["prefix"], case["suffix"], kv_heads=Hkv, tokens=T,
                                                   dtype=dt)
        return st
    B, H = case["B"], case["H"]
    # from a head that looks back over a token or two to one that looks back over hundreds
    u = torch.rand(H, generator=g, device=dev, dtype=torch.float32)
    st["g"] = -torch.exp(math.log(0.7) + (u + torch.arange(H, device=dev)) / H * math.log(0.003 / 0.7))
    if case["op"] == "step":
        st["q"], st["k"], st["v"] = rnd(B, H, D), rnd(B, H, D), rnd(B, H, D)
        st["state"] = rnd(B, H, D, D, dtype=torch.float32)
        S = 1
    else:
        S = case["S"]
        st["q"], st["k"], st["v"] = rnd(B, H, S, D), rnd(B, H, S, D), rnd(B, H, S, D)
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev) if case["ragged"] else None
        st["state"] = rnd(B, H, D, D, dtype=torch.float32) if case["state"] else None
        if case["op"] == "train":
            st["do"] = rnd(B, H, S, D)
            st["dstate"] = rnd(B, H, D, D, dtype=torch.float32) if case["state"] else None
    if own:
        import sharded_causal_softmax_gb300 as sca
        st["plan"] = sca.DecayLinearAttention(B, H, S, D, st["g"], dtype=dt, backward=case["op"] == "train")
    return st


# ------------------------------------------------------------- plain forms

def _chunks(x, n):
    """[B, H, S, D] in 32 bits as [B, H, n, CHUNK, D], zeros behind the last row."""
    B, H, S, D = x.shape
    y = torch.zeros(B, H, n * CHUNK, D, dtype=torch.float32, device=x.device)
    y[:, :, :S] = x
    return y.reshape(B, H, n, CHUNK, D)


def _decays(g, n, device):
    """exp(g * e) in 32 bits for the exponents of a chunk's rows and of whole chunks, from 64-bit powers."""
    g = g.double()
    r = torch.arange(CHUNK, device=device, dtype=torch.float64)
    c = torch.arange(n, device=device, dtype=torch.float64)
    row = torch.exp(g[:, None] * r).float()                                  # [H, C]
    d = r[:, None] - r[None, :]
    intra = torch.where(d >= 0, torch.exp(g[:, None, None] * d.clamp(min=0)), 0.0).float()   # [H, C, C]
    e = c[:, None] - c[None, :] - 1
    inter = torch.where(e >= 0, torch.exp(g[:, None, None] * e.clamp(min=0) * CHUNK), 0.0).float()   # [H, n, n]
    return row, intra, inter


def _forward_sum(x, y, z, g, n):
    """sum_{s <= t} exp(g (t - s)) (x_t . y_s) z_s of chunked x, y, z."""
    B, H, _, _, D = x.shape
    row, intra, inter = _decays(g, n, x.device)
    one = torch.exp(g.double()).float()[None, :, None, None, None]
    near = torch.matmul(torch.matmul(x, y.transpose(-1, -2)) * intra[:, None], z)
    u = torch.matmul((y * row.flip(-1)[:, None, :, None]).transpose(-1, -2), z)     # each chunk's own state
    before = torch.matmul(inter, u.reshape(B, H, n, D * D)).reshape(B, H, n, D, D)
    return near + torch.matmul(x, before) * (row[:, None, :, None] * one)


def _backward_sum(x, y, z, g, n):
    """sum_{s >= t} exp(g (s - t)) (x_t . y_s) z_s of chunked x, y, z."""
    B, H, _, _, D = x.shape
    row, intra, inter = _decays(g, n, x.device)
    one = torch.exp(g.double()).float()[None, :, None, None, None]
    near = torch.matmul(torch.matmul(x, y.transpose(-1, -2)) * intra.transpose(-1, -2)[:, None], z)
    u = torch.matmul((y * row[:, None, :, None]).transpose(-1, -2), z)
    after = torch.matmul(inter.transpose(-1, -2), u.reshape(B, H, n, D * D)).reshape(B, H, n, D, D)
    return near + torch.matmul(x, after) * (row.flip(-1)[:, None, :, None] * one)


def _plain_linear(st):
    q, k, v, g, scale = st["q"], st["k"], st["v"], st["g"], st["scale"]
    B, H, S, D = q.shape
    dev = q.device
    n = -(-S // CHUNK)
    pos = torch.arange(S, device=dev, dtype=torch.float64)
    length = st["lengths"].double() if st["lengths"] is not None else torch.full((B,), float(S), device=dev,
                                                                                 dtype=torch.float64)
    live = (pos < length[:, None])[:, None, :, None]                          # [B, 1, S, 1]
    q, k, v = (torch.where(live, x.float(), 0.0) for x in (q, k, v))
    g64 = g.double()[None, :, None]
    to_here = torch.exp(g64 * (pos + 1)).float()[..., None]                   # exp(g (t + 1)): [1, H, S, 1]
    left = (length[:, None, None] - 1 - pos).clamp(min=0)
    to_end = torch.exp(g64 * left).float()[..., None]                         # exp(g (length - 1 - t)): [B, H, S, 1]
    whole = torch.exp(g64[..., 0] * length[:, None]).float()[..., None, None]  # exp(g length): [B, H, 1, 1]
    qc, kc, vc = _chunks(q, n), _chunks(k, n), _chunks(v, n)

    def flat(x):
        return x.reshape(B, H, n * CHUNK, D)[:, :, :S]

    o = flat(_forward_sum(qc, kc, vc, g, n))
    end = torch.matmul((k * to_end).transpose(-1, -2), v)
    if st["state"] is not None:
        o = o + torch.matmul(q, st["state"]) * to_here
        end = end + st["state"] * whole
    dt = DT[st["case"]["dtype"]]
    out = {"o": (o * scale).to(dt), "state": end}
    if st["case"]["op"] == "prompt":
        return out
    do = torch.where(live, st["do"].float(), 0.0)
    dc = _chunks(do, n)
    dq = flat(_forward_sum(dc, vc, kc, g, n)) * scale
    dk = flat(_backward_sum(vc, dc, qc, g, n)) * scale
    dv = flat(_backward_sum(kc, qc, dc, g, n)) * scale
    first = torch.matmul((q * to_here).transpose(-1, -2), do) * scale
    if st["state"] is not None:
        dq = dq + torch.matmul(do, st["state"].transpose(-1, -2)) * to_here * scale
    if st["dstate"] is not None:
        dk = dk + torch.where(live, torch.matmul(v, st["dstate"].transpose(-1, -2)) * to_end, 0.0)
        dv = dv + torch.where(live, torch.matmul(k, st["dstate"]) * to_end, 0.0)
        first = first + st["dstate"] * whole
    out.update(dq=dq.to(dt), dk=dk.to(dt), dv=dv.to(dt))
    if st["state"] is not None:
        out["dstate"] = first
    return out


def _plain_step(st):
    k, v, q = st["k"].float(), st["v"].float(), st["q"].float()
    lam = torch.exp(st["g"].double()).float()[None, :, None, None]
    st["state"].copy_(st["state"] * lam + k[..., :, None] * v[..., None, :])
    o = torch.matmul(q[..., None, :], st["state"])[..., 0, :] * st["scale"]
    return {"o": o.to(DT[st["case"]["dtype"]]), "state": st["state"]}


def _plain_decode(st):
    c = st["case"]
    B, Hkv, T, D, R = c["B"], c["Hkv"], c["T"], c["D"], c["group"] * c["T"]
    q = st["q"].float().reshape(B, Hkv, R, D)
    kp, vp, ks, vs = (st[x].float() for x in ("kp", "vp", "ks", "vs"))
    j = torch.arange(c["suffix"], device=q.device)
    t = torch.arange(T, device=q.device).repeat(c["group"])                     # the token of each row
    last = st["lengths"][:, None].long() - (T - 1 - t)[None, :]                  # [B, R]
    live = (j < st["lengths"][:, None])[:, None, :, None]
    vs = torch.where(live, vs, 0.0)
    qh = q.transpose(0, 1).reshape(Hkv, B * R, D)
    sp = (torch.matmul(qh, kp.transpose(-1, -2)) * st["scale"]).reshape(Hkv, B, R, -1).transpose(0, 1)
    ss = torch.matmul(q, ks.transpose(-1, -2)) * st["scale"]
    ss = torch.where((j < last[..., None])[:, None], ss, float("-inf"))
    m = torch.maximum(sp.amax(-1), ss.amax(-1))
    pp, ps = torch.exp(sp - m[..., None]), torch.exp(ss - m[..., None])
    total = pp.sum(-1) + ps.sum(-1)
    op = torch.matmul(pp.transpose(0, 1).reshape(Hkv, B * R, -1), vp).reshape(Hkv, B, R, D).transpose(0, 1)
    o = (op + torch.matmul(ps, vs)) / total[..., None]
    return {"o": o.reshape(B, Hkv * c["group"], T, D).to(DT[c["dtype"]]),
            "lse": (m + torch.log(total)).reshape(B, Hkv * c["group"], T)}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"step": _plain_step, "decode": _plain_decode}.get(op, _plain_linear)(state)
    plan = state["plan"]
    if op == "step":
        o = plan.step(state["q"], state["k"], state["v"], state["state"])
        return {"o": o, "state": state["state"]}
    if op == "decode":
        o, lse = plan.decode(state["q"], state["kp"], state["vp"], state["ks"], state["vs"], state["lengths"])
        return {"o": o, "lse": lse}
    o, end = plan.forward(state["q"], state["k"], state["v"], state=state["state"], lengths=state["lengths"])
    out = {"o": o, "state": end}
    if op == "train":
        dq, dk, dv, first = plan.backward(state["do"], dstate=state["dstate"])
        out.update(dq=dq, dk=dk, dv=dv)
        if state["state"] is not None:
            out["dstate"] = first
    return out


def work(case):
    """Inputs read once, outputs written once; products of the chunked form with chunks of CHUNK rows (linear), of the visible keys (decode)."""
    D, eb = case["D"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "decode":
        rows = case["B"] * case["Hkv"] * case["group"] * case["T"]
        own_keys = sum(_lengths(case))
        keys = case["Hkv"] * (case["prefix"] + own_keys)
        seen = rows * case["prefix"] + case["Hkv"] * case["group"] * case["T"] * own_keys
        return {"bytes": 2 * keys * D * eb + 2 * rows * D * eb + 4 * rows, "flops": 4 * seen * D}
    B, H = case["B"], case["H"]
    if case["op"] == "step":
        return {"bytes": B * H * (2 * D * D * 4 + 4 * D * eb) + 4 * H, "flops": 5 * B * H * D * D}
    live = H * sum(_lengths(case))
    full = B * H * case["S"]
    states = B * H * D * D * 4
    per_row = 4 * D * D + 4 * D * min(CHUNK, case["S"])
    if case["op"] == "prompt":
        return {"bytes": (3 * live + full) * D * eb + states * (1 + case["state"]), "flops": live * per_row}
    return {"bytes": (4 * live + 4 * full) * D * eb + states * (1 + 3 * case["state"]), "flops": live * 3 * per_row}


# ------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(st)
    q, k, v = (st[x].double() for x in ("q", "k", "v"))
    lam = torch.exp(st["g"].double())[None, :, None, None]
    if case["op"] == "step":
        s = lam * st["state"].double() + torch.einsum("bhd,bhe->bhde", k, v)
        return {"o": torch.einsum("bhd,bhde->bhe", q, s) * st["scale"], "state": s}
    B, H, S, D = q.shape
    if st["lengths"] is None:
        alive = torch.ones(S, B, 1, 1, 1, dtype=torch.bool, device=q.device)
    else:
        alive = (torch.arange(S, device=q.device)[:, None] < st["lengths"].long())[:, :, None, None, None]
    s = torch.zeros(B, H, D, D, dtype=torch.float64, device=q.device)
    if st["state"] is not None:
        s = st["state"].double()
    o, dq = torch.zeros_like(q), torch.zeros_like(q)
    do = st["do"].double() if case["op"] == "train" else None
    every = st["lengths"] is None
    for t in range(S):
        new = torch.baddbmm((lam * s).reshape(B * H, D, D), k[:, :, t].reshape(B * H, D, 1),
                            v[:, :, t].reshape(B * H, 1, D)).reshape(B, H, D, D)
        s = new if every else torch.where(alive[t], new, s)
        o[:, :, t] = torch.matmul(q[:, :, t, None], s)[:, :, 0]
        if do is not None:
            dq[:, :, t] = torch.matmul(s, do[:, :, t, :, None])[..., 0]
    here = alive.reshape(S, B).T[:, None, :, None]
    out = {"o": torch.where(here, o, 0.0) * st["scale"], "state": s}
    if case["op"] == "prompt":
        return out
    # the loss's derivative by the state, from the last row back; `s` is by the state after the row
    s = torch.zeros(B, H, D, D, dtype=torch.float64, device=q.device)
    if st["dstate"] is not None:
        s = st["dstate"].double()
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in range(S - 1, -1, -1):
        at = torch.baddbmm(s.reshape(B * H, D, D), q[:, :, t].reshape(B * H, D, 1),
                           do[:, :, t].reshape(B * H, 1, D), alpha=st["scale"]).reshape(B, H, D, D)
        dk[:, :, t] = torch.matmul(at, v[:, :, t, :, None])[..., 0]
        dv[:, :, t] = torch.matmul(k[:, :, t, None], at)[:, :, 0]
        s = lam * at if every else torch.where(alive[t], lam * at, s)
    out.update(dq=torch.where(here, dq, 0.0) * st["scale"], dk=torch.where(here, dk, 0.0),
               dv=torch.where(here, dv, 0.0))
    if st["state"] is not None:
        out["dstate"] = s
    return out


def _exact_decode(st):
    c = st["case"]
    H, T = c["Hkv"] * c["group"], c["T"]
    o = torch.zeros(c["B"], H, T, c["D"], dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros(c["B"], H, T, dtype=torch.float64, device=st["q"].device)
    lengths = st["lengths"].tolist()
    for h in range(c["Hkv"]):
        kp, vp = st["kp"][h].double(), st["vp"][h].double()
        mine = slice(h * c["group"], (h + 1) * c["group"])
        for b in range(c["B"]):
            for t in range(T):
                n = max(0, lengths[b] - (T - 1 - t))
                keys = torch.cat([kp, st["ks"][b, h, :n].double()])
                values = torch.cat([vp, st["vs"][b, h, :n].double()])
                x = st["q"][b, mine, t].double() @ keys.T * st["scale"]
                lse[b, mine, t] = torch.logsumexp(x, -1)
                o[b, mine, t] = torch.softmax(x, -1) @ values
    return {"o": o, "lse": lse}
