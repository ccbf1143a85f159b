"""Decode attention over long caches whose row maxima grow again and again
within one CTA's keys, in any of the four groups of 32 keys of a tile, in rows
of one warp at different places: what the running output and the weights so
far are scaled by must reach both each time.

The scores rise in steps of 9.5 powers of two up to a peak, tile after tile,
then start from below; a key n steps below the peak has values 2^(9 min(n, 10))
as large, so that every step matters in the result: a step that is lost, or
taken from numbers of before the last one, puts a row off by hundreds of times
its own size.

Bounds as for any decode step, o off by (2 es + n 2^-23 + 2^-20) A for n keys
with A the sum over the values' magnitudes and es a score's error, plus 2^-8 A
each time a weight is rounded: when it is made and at up to three later steps
in its tile; and for each of up to 40 steps the rounding of a difference of at
most 400 powers of two, 400 2^-24 ln 2 of A."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

PERIOD = 6   # tiles from one peak to the next: a CTA's part of the long cases holds at least that many


@pytest.fixture(scope="module")
def sca():
    import sharded_causal_softmax_gb300 as m
    from sharded_causal_softmax_gb300 import build
    build.build()
    return m


def steps_below(n, turn):
    """Steps from each of n keys to the next peak: tile i grows at the groups of 32 in the bits of i + turn."""
    tiles = -(-n // 128)
    up = torch.tensor([[(i + turn) >> h & 1 for h in range(4)] for i in range(tiles)])
    left = torch.zeros_like(up)
    for first in range(0, tiles, PERIOD):
        own = up[first:first + PERIOD].reshape(-1)
        left[first:first + PERIOD] = (own.sum() - own.cumsum(0)).reshape(-1, 4)
    return left.reshape(-1).repeat_interleave(32)[:n]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,group,kind", [(64, 4, "prefix"), (2, 3, "prefix"), (90, 3, "prefix"), (2, 3, "suffix")])
def test_maxima_that_grow_within_a_part(sca, B, group, kind, D):
    """Two row tiles on the same keys; one, its keys in turn on two streams; both kinds; a suffix."""
    n = 152 * 7 * 128 + 37 if kind == "prefix" else 152 * 4 * 128 + 5
    g = torch.Generator(device="cuda").manual_seed(B + D)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    u = torch.linalg.qr(rnd(D, 2))[0].T                                        # two directions that rows lean on
    below = torch.stack([steps_below(n, 0), steps_below(n, 5)]).cuda()           # [2, n]
    k = -9.5 * math.log(2) * below.T.float() @ u + 0.05 * rnd(n, D)
    size = torch.exp2(9.0 * below.clamp(max=10))
    v = rnd(n, D) * torch.cat([size[0][:, None].expand(n, D // 2), size[1][:, None].expand(n, D // 2)], 1)
    q = math.sqrt(D) * u[torch.arange(B * group, device="cuda") % 2] + 0.05 * rnd(B * group, D)
    q, k, v = (t.bfloat16() for t in (q, k, v))
    if kind == "prefix":
        lengths = [n] * B
        args = (q.view(B, group, 1, D), k[None], v[None], None, None, None)
        plan = sca.SharedPrefixAttention(B, group, D, n, 0, kv_heads=1)
    else:
        lengths = [n, n - 1000]
        args = (q.view(B, group, 1, D), None, None, *(t.expand(B, 1, n, D).contiguous() for t in (k, v)),
                torch.tensor(lengths, dtype=torch.int32, device="cuda"))
        plan = sca.SharedPrefixAttention(B, group, D, 0, n, kv_heads=1)
    for t in (plan.o, plan.lse, plan._ws):
        t.fill_(float("nan"))
    o, lse = (t.clone() for t in plan.decode(*args))
    assert plan.read_status() == 0
    assert all(torch.equal(a, b) for a, b in zip((o, lse), plan.decode(*args)))

    s = q.double() @ k.double().T * plan.scale
    end = torch.tensor(lengths, device="cuda").repeat_interleave(group)
    s = torch.where(torch.arange(n, device="cuda") < end[:, None], s, -math.inf)
    top = s.amax(1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(1, keepdim=True)
    ref, mag, rl = (p @ v.double() / total, p @ v.double().abs() / total, (top + total.log())[:, 0])
    assert below.max() * 9.5 + 8 < 400 and below.max() <= 40
    es = D * 2.0 ** -23 * float(q.double().norm(dim=1).max() * k.double().norm(dim=1).max()) * plan.scale + 2.0 ** -21
    err = 2 * es + n * 2.0 ** -23 + 2.0 ** -20 + 4 * 2.0 ** -8 + 40 * 400 * 2.0 ** -24 * math.log(2)
    d = (o.double().view(-1, D) - ref).abs()
    bound = 1.01 * 2.0 ** -8 * ref.abs() + err * mag
    assert (d <= bound).all(), f"o: worst {(d / bound).max().item():.2f} of the bound"
    dl = (lse.double().view(-1) - rl).abs()
    lb = es + n * 2.0 ** -24 + 2.0 ** -20 + 40 * 400 * 2.0 ** -24 * math.log(2) + 2.0 ** -23 * rl.abs()
    assert (dl <= lb).all(), f"lse: worst {(dl / lb).max().item():.2f} of the bound"
