"""Decaying linear attention and shared-prefix decoding at the edges of what
the entry points take."""
import math

import pytest
import torch

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
