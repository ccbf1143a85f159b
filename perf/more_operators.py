"""Cases for measuring the operators that give attention its positions and
serve it from a paged cache, and their plain forms.

Rotary positions.  With f_i the frequency of pair i of the first ``rd``
features and p the row's position, both numbers of the pair are turned:

    y_a = a (x_a cos(p f_i) - x_b sin(p f_i)),   y_b = a (x_a sin(p f_i) + x_b cos(p f_i))

(a: 1, or what the scaling for long contexts asks for; pairs (i, i + rd / 2)
in the "half" layout, (2 i, 2 i + 1) in the "interleaved" one; the other
features stay).  ``rotate``: queries and keys; ``rotate_train``: those, and the
gradients by the same rows.

A cache of keys and values in pages, [pages, heads, page, D], of which request
b holds rows 0, 1, ... of its own through a table of page numbers:
``append`` writes the keys (turned to their positions on the way) and values of
new rows behind the ``lengths`` that are there, and turns the queries;
``attend`` is the attention of drafted tokens over it: node t of a request's
tree sees its first ``lengths`` rows and those of the nodes in t's mask, which
follow them; ``accept`` moves the rows of the nodes that were right to where
the next call expects them.  Nodes at or past ``counts`` are padding.

Where ``own`` is false ``run`` computes them with elementary torch operations.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LOW, HIGH = 1.0, 32.0   # turns over the trained length between which the "ramp" goes from scaled to unscaled


def listed():
    return [
        # a chat turn's short prompt on a small model: latency
        dict(name="rotate_short", op="rotate", B=1, H=8, Hkv=8, S=77, D=64, rd=64, layout="half", scaling="none",
             factor=1.0, given=False, dtype="bf16"),
        # a numerics run in full precision, part of each head turned, odd lengths at given positions
        dict(name="rotate_f32", op="rotate_train", B=3, H=12, Hkv=4, S=1001, D=64, rd=32, layout="interleaved",
             scaling="linear", factor=4.0, given=True, dtype="f32"),
        # the repository's training step, 16 heads of 32K rows, for a context eight times as long as the trained one
        dict(name="rotate_32k", op="rotate_train", B=1, H=16, Hkv=16, S=32768, D=128, rd=128, layout="half",
             scaling="ramp", factor=8.0, given=False, dtype="bf16"),
        # the drafted tokens of a full batch, at the positions of their tree, the repository's 32 heads on 8
        dict(name="append_drafts", op="append", B=64, H=32, Hkv=8, T=8, D=128, rd=128, layout="half", scaling="base",
             factor=4.0, given=True, keys=2048, page=16, ragged=False, dtype="bf16"),
        # a batch of prompts of mixed lengths behind what is there, half of each head turned
        dict(name="append_prompts", op="append", B=8, H=32, Hkv=8, T=2049, D=128, rd=64, layout="interleaved",
             scaling="none", factor=1.0, given=False, keys=513, page=64, ragged=True, dtype="bf16"),
        # one request's next token: latency
        dict(name="attend_one", op="attend", B=1, Hkv=8, group=4, T=1, keys=1000, D=128, page=16, tree=False,
             ragged=False, dtype="bf16"),
        # a batch's drafts verified, an odd group of heads, mixed lengths
        dict(name="attend_verify", op="attend", B=13, Hkv=4, group=5, T=24, keys=8191, D=128, page=64, tree=True,
             ragged=True, dtype="bf16"),
        # a small model kept in 32 bits, every head its own keys
        dict(name="attend_f32", op="attend", B=5, Hkv=8, group=1, T=9, keys=1003, D=64, page=32, tree=True,
             ragged=True, dtype="f32"),
        # a full batch of long contexts, one token each: the cache streams through the card
        dict(name="attend_long", op="attend", B=32, Hkv=8, group=4, T=1, keys=32768, D=128, page=64, tree=False,
             ragged=False, dtype="bf16"),
        # wide trees over long contexts: products as much as bytes
        dict(name="attend_wide", op="attend", B=16, Hkv=8, group=4, T=64, keys=16384, D=128, page=128, tree=True,
             ragged=False, dtype="bf16"),
        # one request's accepted drafts: latency
        dict(name="accept_one", op="accept", B=1, Hkv=8, T=16, keys=500, D=64, page=16, dtype="bf16"),
        # a full batch's
        dict(name="accept_batch", op="accept", B=256, Hkv=8, T=64, keys=1000, D=128, page=32, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _angles(rng, D):
    scaling = rng.choice(("none", "linear", "base", "ramp"))
    return dict(rd=rng.choice((D, D, D // 2, D // 4)), layout=rng.choice(("half", "interleaved")), scaling=scaling,
                factor=1.0 if scaling == "none" else float(rng.choice((2, 4, 8, 32))), given=rng.random() < 0.5)


def draw(rng):
    op = rng.choice(("rotate", "rotate_train", "append", "attend", "attend", "accept"))
    D = rng.choice((64, 128))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op.startswith("rotate"):
        B, Hkv, group = _log_int(rng, 1, 16), _log_int(rng, 1, 8), _log_int(rng, 1, 8)
        heads = Hkv * (group + 1)
        cap = (1 << 26 if dtype == "bf16" else 1 << 25) // D
        S = _log_int(rng, 1, max(1, min(32768, cap // (B * heads))))
        return dict(op=op, B=B, H=Hkv * group, Hkv=Hkv, S=S, D=D, dtype=dtype, **_angles(rng, D))
    page = rng.choice((16, 32, 64, 128))
    Hkv = _log_int(rng, 1, 8)
    if op == "append":
        B, group = _log_int(rng, 1, 64), _log_int(rng, 1, 8)
        T = _log_int(rng, 1, max(1, min(4096, (1 << 25) // (B * Hkv * (group + 2) * D))))
        keys = _log_int(rng, 1, max(1, min(4096, (1 << 19) // (B * Hkv))))
        return dict(op=op, B=B, H=Hkv * group, Hkv=Hkv, T=T, D=D, keys=keys, page=page, ragged=rng.random() < 0.5,
                    dtype=dtype, **_angles(rng, D))
    if op == "accept":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, Hkv=Hkv, T=_log_int(rng, 1, 64), keys=_log_int(rng, 1, 1024), D=D, page=page,
                    dtype=dtype)
    B, group, T = _log_int(rng, 1, 64), _log_int(rng, 1, 8), rng.choice((1, 1, _log_int(rng, 2, 64)))
    rows = B * Hkv * group * T
    most = 1 << 28 if dtype == "bf16" else 1 << 23   # query rows x keys
    keys = _log_int(rng, 1, max(1, min(65536, most // rows, (1 << 22) // (B * Hkv))))
    return dict(op=op, B=B, Hkv=Hkv, group=group, T=T, keys=keys, D=D, page=page, tree=T > 1 and rng.random() < 0.8,
                ragged=rng.random() < 0.6, dtype=dtype)


# --------------------------------------------------------------- the cases' own numbers, the same for every seed

def _lengths(case):
    """Rows that each request holds before the call."""
    rng = random.Random(7 * case["B"] + case["keys"])
    if not case.get("ragged", True):
        return [case["keys"]] * case["B"]
    return [case["keys"]] + [rng.randint(0, case["keys"]) for _ in range(case["B"] - 1)]


def _counts(case):
    """New rows of each request; the first brings all of them."""
    rng = random.Random(11 * case["B"] + case["T"])
    if not case.get("ragged", True):
        return [case["T"]] * case["B"]
    return [case["T"]] + [rng.randint(0, case["T"]) for _ in range(case["B"] - 1)]


def _accepted(case):
    """Nodes of each request that were right: mostly few."""
    rng = random.Random(13 * case["B"] + case["T"])
    return [min(case["T"], 1 + int(rng.expovariate(0.4))) for _ in range(case["B"])]


def _frequencies(case):
    """(radians a position of every pair, the factor on the turned numbers), in 64 bits."""
    rd, s = case["rd"], case["factor"]
    base = 10000.0
    if case["scaling"] == "base" and rd > 2:
        base *= s ** (rd / (rd - 2))
    f = [base ** (-2.0 * i / rd) for i in range(rd // 2)]
    if case["scaling"] == "linear":
        f = [x / s for x in f]
    if case["scaling"] == "ramp":
        keep = [min(1.0, max(0.0, (4096 * x / (2 * math.pi) - LOW) / (HIGH - LOW))) for x in f]
        return [x * (g + (1 - g) / s) for x, g in zip(f, keep)], 0.1 * math.log(s) + 1.0
    return f, 1.0


# ----------------------------------------------------------------------------------------------------- inputs

def _trees(case, seed, device):
    """(int64 masks of what each node sees, itself among it; depths) of random trees, one a request."""
    rng = random.Random(seed)
    masks, depths = [], []
    for _ in range(case["B"]):
        m, d = [], []
        for t in range(case["T"]):
            p = rng.randint(max(0, t - 6), t - 1) if t else -1
            m.append((m[p] if t else 0) | 1 << t)
            d.append(d[p] + 1 if t else 0)
        masks.append([x - (1 << 64) if x >> 63 else x for x in m])
        depths.append(d)
    return torch.tensor(masks, dtype=torch.int64, device=device), torch.tensor(depths, dtype=torch.int32, device=device)


def _own_angles(case, device):
    import sharded_causal_softmax_gb300 as sca
    scaling = {"none": None, "linear": ("linear", case["factor"]), "base": ("base", case["factor"]),
               "ramp": ("ramp", case["factor"], 4096, LOW, HIGH)}[case["scaling"]]
    return sca.RotaryAngles(case["rd"], base=10000.0, layout=case["layout"], scaling=scaling, device=device)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[case["dtype"]]

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    st = {"case": case}
    op, B, D, Hkv = case["op"], case["B"], case["D"], case["Hkv"]
    if op.startswith("rotate"):
        H, S = case["H"], case["S"]
        st["q"], st["k"] = rnd(B, H, S, D), rnd(B, Hkv, S, D)
        if op == "rotate_train":
            st["dq"], st["dk"] = rnd(B, H, S, D), rnd(B, Hkv, S, D)
        st["positions"] = None
        if case["given"]:   # parts of long documents
            rng = random.Random(seed)
            first = ints([rng.randint(0, 1 << 20) for _ in range(B)])
            st["positions"] = first[:, None] + torch.arange(S, dtype=torch.int32, device=dev)
        if own:
            import sharded_causal_softmax_gb300 as sca
            st["plan"] = sca.RotaryPositions(B, H, S, D, _own_angles(case, dev), kv_heads=Hkv, dtype=dt,
                                             backward=op == "rotate_train")
        return st
    T, page = case["T"], case["page"]
    lengths = _lengths(case)
    each = -(-(case["keys"] + T) // page)      # pages of a request
    pages = B * each + 3
    # a pool that has been in use for a while: any page anywhere, old rows in all of them
    st["table"] = torch.randperm(pages, generator=g, device=dev)[:B * each].to(torch.int32).reshape(B, each)
    st["k_pages"], st["v_pages"] = rnd(pages, Hkv, page, D), rnd(pages, Hkv, page, D)
    st["lengths"] = ints(lengths)
    if op == "append":
        H = case["H"]
        st["counts"] = ints(_counts(case)) if case["ragged"] else None
        qkv = rnd(B, T, H + 2 * Hkv, D).transpose(1, 2)       # one projection's output
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        st["positions"] = None
        if case["given"]:   # a drafted token lies behind its parent; the documents go on from elsewhere
            depth = torch.arange(T, dtype=torch.int32, device=dev) // 2
            st["positions"] = (st["lengths"] + 5000)[:, None] + depth
    elif op == "attend":
        st["counts"] = ints(_counts(case)) if case["ragged"] else None
        st["q"] = rnd(B, Hkv * case["group"], T, D)
        st["tree"] = _trees(case, seed, dev)[0] if case["tree"] else None
    else:
        rng = random.Random(seed)
        st["path"] = ints([sorted(rng.sample(range(T), n)) + [0] * (T - n) for n in _accepted(case)])
        st["accepted"] = ints(_accepted(case))
    if own:
        import sharded_causal_softmax_gb300 as sca
        angles = _own_angles(case, dev) if op == "append" else None
        st["cache"] = sca.PagedKVCache(pages, Hkv, D, page=page, dtype=dt, angles=angles,
                                       pools=(st["k_pages"], st["v_pages"]))
        H = Hkv * case["group"] if op == "attend" else case["H"] if op == "append" else Hkv
        st["plan"] = sca.PagedTreeAttention(st["cache"], B, H, tokens=T, keys=each * page)
    return st


# ------------------------------------------------------------------------------------------------- plain forms

def _turns(case, positions):
    """cos and sin, 32 bits, [..., rd / 2], of positions [...]: the angles of far positions need 64."""
    f, a = _frequencies(case)
    x = positions.double()[..., None] * torch.tensor(f, dtype=torch.float64, device=positions.device)
    return (torch.cos(x) * a).float(), (torch.sin(x) * a).float()


def _rotated(x, cos, sin, case, back=False):
    """x [B, H, S, D] turned (``back``: by the transposed matrix); cos, sin [B or 1, 1, S, rd / 2]."""
    rd = case["rd"]
    y = x.float()
    if case["layout"] == "half":
        u, w = y[..., :rd // 2], y[..., rd // 2:rd]
    else:
        u, w = y[..., 0:rd:2], y[..., 1:rd:2]
    s = -sin if back else sin
    u, w = u * cos - w * s, u * s + w * cos
    if case["layout"] == "half":
        turned = torch.cat([u, w], -1)
    else:
        turned = torch.stack([u, w], -1).flatten(-2)
    return torch.cat([turned, y[..., rd:]], -1).to(x.dtype)


def _plain_rotate(st):
    c = st["case"]
    positions = st["positions"]
    if positions is None:
        positions = torch.arange(c["S"], device=st["q"].device)[None]
    cos, sin = (x[:, None] for x in _turns(c, positions))
    out = {"q": _rotated(st["q"], cos, sin, c), "k": _rotated(st["k"], cos, sin, c)}
    if c["op"] == "rotate_train":
        out.update(dq=_rotated(st["dq"], cos, sin, c, back=True), dk=_rotated(st["dk"], cos, sin, c, back=True))
    return out


def _places(st, slots):
    """(page numbers, rows in them) of slots [B, n]."""
    page = st["case"]["page"]
    return torch.gather(st["table"].long(), 1, slots // page), slots % page


def _plain_append(st):
    c = st["case"]
    t = torch.arange(c["T"], device=st["q"].device)
    slots = st["lengths"].long()[:, None] + t
    positions = slots if st["positions"] is None else st["positions"]
    cos, sin = (x[:, None] for x in _turns(c, positions))
    at, row = _places(st, slots)
    live = torch.ones_like(slots, dtype=torch.bool) if st["counts"] is None else t < st["counts"][:, None]
    live = live[:, :, None, None]
    new = {"k_pages": _rotated(st["k"], cos, sin, c), "v_pages": st["v"]}
    for name, x in new.items():   # padding puts back what is there
        pool = st[name]
        pool[at, :, row] = torch.where(live, x.transpose(1, 2), pool[at, :, row])
    q = torch.where(live.transpose(1, 2), _rotated(st["q"], cos, sin, c), 0.0)
    return {"q": q.to(DT[c["dtype"]]), "k": st["k_pages"], "v": st["v_pages"]}


def _plain_attend(st):
    c = st["case"]
    B, Hkv, T, D, R = c["B"], c["Hkv"], c["T"], c["D"], c["group"] * c["T"]
    table = st["table"].long()

    def rows(pool):   # [B, Hkv, rows of all pages, D]
        return pool[table].transpose(1, 2).reshape(B, Hkv, -1, D).float()

    k, v = rows(st["k_pages"]), rows(st["v_pages"])
    n = k.shape[2]
    node = torch.arange(n, device=k.device) - st["lengths"].long()[:, None]               # [B, n]: which node a key is
    t = torch.arange(T, device=k.device)
    counts = torch.full((B,), T, device=k.device) if st["counts"] is None else st["counts"].long()
    if st["tree"] is None:
        seen = node[:, None] <= t[:, None]
    else:
        bit = (st["tree"][:, :, None] >> node.clamp(0, T - 1)[:, None]) & 1
        seen = (node < 0)[:, None] | (bit == 1)
    seen &= (node < counts[:, None])[:, None] & (t < counts[:, None])[:, :, None]         # [B, T, n]
    s = torch.matmul(st["q"].float().reshape(B, Hkv, R, D), k.transpose(-1, -2)) / math.sqrt(D)
    s = torch.where(seen[:, None, None], s.reshape(B, Hkv, c["group"], T, n), float("-inf")).reshape(B, Hkv, R, n)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return {"o": o.reshape(B, Hkv * c["group"], T, D).to(DT[c["dtype"]]),
            "lse": (m + torch.log(total)).reshape(B, Hkv * c["group"], T)}


def _plain_accept(st):
    c = st["case"]
    i = torch.arange(c["T"], device=st["path"].device)
    first = st["lengths"].long()[:, None]
    live = (i < st["accepted"][:, None])[:, :, None, None]
    here, there = _places(st, first + i), _places(st, first + st["path"].long())
    for pool in (st["k_pages"], st["v_pages"]):
        pool[here[0], :, here[1]] = torch.where(live, pool[there[0], :, there[1]], pool[here[0], :, here[1]])
    return {"k": st["k_pages"], "v": st["v_pages"], "lengths": st["lengths"] + st["accepted"]}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "accept": _plain_accept}.get(op, _plain_rotate)(state)
    plan = state["plan"]
    if op == "append":
        q = plan.append(state["q"], state["k"], state["v"], state["table"], state["lengths"], counts=state["counts"],
                        positions=state["positions"])
        return {"q": q, "k": state["k_pages"], "v": state["v_pages"]}
    if op == "attend":
        o, lse = plan.attend(state["q"], state["table"], state["lengths"], counts=state["counts"], tree=state["tree"])
        return {"o": o, "lse": lse}
    if op == "accept":
        lengths = plan.accept(state["table"], state["lengths"], state["path"], state["accepted"])
        return {"k": state["k_pages"], "v": state["v_pages"], "lengths": lengths}
    q, k = plan.forward(state["q"], state["k"], positions=state["positions"])
    out = {"q": q, "k": k}
    if op == "rotate_train":
        out["dq"], out["dk"] = plan.backward(state["dq"], state["dk"])
    return out


def work(case):
    """Inputs read once, outputs written once: of the pools, the rows that a call reads or writes."""
    D, eb, op, B, Hkv = case["D"], 2 if case["dtype"] == "bf16" else 4, case["op"], case["B"], case["Hkv"]
    if op.startswith("rotate"):
        rows = B * case["S"] * (case["H"] + Hkv) * (2 if op == "rotate_train" else 1)
        return {"bytes": 2 * rows * D * eb + (4 * B * case["S"] if case["given"] else 0), "flops": 3 * rows * case["rd"]}
    if op == "append":
        rows = sum(_counts(case)) * (case["H"] + 2 * Hkv)
        pad = (B * case["T"] - sum(_counts(case))) * case["H"]
        return {"bytes": (2 * rows + pad) * D * eb + 4 * B * case["T"] * case["given"],
                "flops": 3 * sum(_counts(case)) * (case["H"] + Hkv) * case["rd"]}
    if op == "accept":
        return {"bytes": 4 * Hkv * D * eb * sum(_accepted(case)) + 4 * B * case["T"], "flops": 0}
    lengths, counts = _lengths(case), _counts(case)
    keys = Hkv * sum(n + c for n, c in zip(lengths, counts) if c)
    rows = B * Hkv * case["group"] * case["T"]
    seen = Hkv * case["group"] * sum(c * (n + c / 2) for n, c in zip(lengths, counts))
    return {"bytes": 2 * keys * D * eb + 2 * rows * D * eb + 4 * rows, "flops": 4 * seen * D}


# --------------------------------------------------------------------------------- the definitions in 64 bits

def _exact_turned(x, angle, a, rd, half, sign=1.0):
    """x [..., S, D] as complex numbers times a e^(i sign angle), angle [..., S, rd / 2]."""
    y = x.double().clone()
    i = torch.arange(rd // 2, device=x.device)
    re, im = (i, i + rd // 2) if half else (2 * i, 2 * i + 1)
    z = torch.complex(y[..., re], y[..., im]) * torch.polar(torch.full_like(angle, a), sign * angle)
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_angle(case, positions):
    """([..., rd / 2] angles, the factor)."""
    rd, s = case["rd"], case["factor"]
    i = torch.arange(rd // 2, dtype=torch.float64, device=positions.device)
    base = torch.tensor(10000.0, dtype=torch.float64, device=positions.device)
    if case["scaling"] == "base" and rd > 2:
        base = base * s ** (rd / (rd - 2))
    f = torch.exp(-torch.log(base) * 2 * i / rd)
    a = 1.0
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "ramp":
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        f, a = keep * f + (1 - keep) * f / s, 1.0 + math.log(s) / 10
    return positions.double()[..., None] * f, a


def exact(case, seed):
    st = prepare(case, seed)
    op, half = case["op"], case.get("layout") == "half"
    if op.startswith("rotate"):
        p = torch.arange(case["S"], device=st["q"].device).expand(case["B"], -1)
        angle, a = _exact_angle(case, p if st["positions"] is None else st["positions"])
        out = {}
        for name in ("q", "k", "dq", "dk"):
            if name in st:
                sign = -1.0 if name.startswith("d") else 1.0
                out[name] = torch.stack([_exact_turned(st[name][b], angle[b], a, case["rd"], half, sign)
                                         for b in range(case["B"])])
        return out
    lengths, table = st["lengths"].tolist(), st["table"].tolist()
    k, v = st["k_pages"].double(), st["v_pages"].double()
    page = case["page"]
    counts = [case["T"]] * case["B"]
    if st.get("counts") is not None:
        counts = st["counts"].tolist()
    if op == "append":
        q = torch.zeros(case["B"], case["H"], case["T"], case["D"], dtype=torch.float64, device=k.device)
        for b, (n, c) in enumerate(zip(lengths, counts)):
            slots = torch.arange(n, n + c, device=k.device)
            angle, a = _exact_angle(case, slots if st["positions"] is None else st["positions"][b, :c])
            q[b, :, :c] = _exact_turned(st["q"][b, :, :c], angle, a, case["rd"], half)
            at = st["table"][b].long()[slots // page]
            k[at, :, slots % page] = _exact_turned(st["k"][b, :, :c], angle, a, case["rd"], half).transpose(0, 1)
            v[at, :, slots % page] = st["v"][b, :, :c].double().transpose(0, 1)
        return {"q": q, "k": k, "v": v}
    if op == "accept":
        path, accepted = st["path"].tolist(), st["accepted"].tolist()
        for pool in (k, v):
            old = pool.clone()
            src, dst = [], []
            for b, n in enumerate(lengths):
                for i in range(accepted[b]):
                    src.append(table[b][(n + path[b][i]) // page] * page + (n + path[b][i]) % page)
                    dst.append(table[b][(n + i) // page] * page + (n + i) % page)
            s, d = torch.tensor(src, device=k.device), torch.tensor(dst, device=k.device)
            pool[d // page, :, d % page] = old[s // page, :, s % page]
        return {"k": k, "v": v, "lengths": st["lengths"] + st["accepted"]}
    B, H, T, D = st["q"].shape
    del k, v
    o = torch.zeros(B, H, T, D, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((B, H, T), float("-inf"), dtype=torch.float64, device=st["q"].device)
    group = case["group"]
    for b, (n, c) in enumerate(zip(lengths, counts)):
        if not c:
            continue
        mine = st["table"][b, :-(-(n + c) // page)].long()
        keys, values = (st[x][mine].transpose(0, 1).reshape(case["Hkv"], -1, D)[:, :n + c].double()
                        for x in ("k_pages", "v_pages"))
        hidden = torch.ones(c, c, dtype=torch.bool).triu(1)
        if st["tree"] is not None:
            words = st["tree"][b, :c].tolist()
            hidden = torch.tensor([[not (w >> u) & 1 for u in range(c)] for w in words])
        x = torch.einsum("hgtd,hjd->hgtj", st["q"][b].double().reshape(case["Hkv"], group, T, D)[:, :, :c], keys)
        x = x / math.sqrt(D)
        x[..., n:].masked_fill_(hidden.to(x.device), float("-inf"))
        lse[b, :, :c] = torch.logsumexp(x, -1).reshape(H, c)
        o[b, :, :c] = torch.einsum("hgtj,hjd->hgtd", torch.softmax(x, -1), values).reshape(H, c, D)
    return {"o": o, "lse": lse}
