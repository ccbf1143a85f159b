"""Entries outside the pool, tables that end too early and offsets beyond 32 bits,
for the kernels of many query rows (40 to 200 of a key/value head), each of which
looks pages up by itself."""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_paged import DT, HALF, Setup, code_of, compare, ints, sca  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = [
    # dtype, algo, group, T, older rows
    ("f32", "auto", 8, 8, [520, 600, 555]), ("f32", "auto", 8, 5, [3000, 1000, 0]), ("bf16", "tc", 10, 6, [520, 600, 556]),
    ("bf16", "tc", 25, 8, [3000, 1000, 0]), ("bf16", "tc", 1, 200, [3000, 1000, 400]),
]
IDS = ["fp32_tiles", "fp32_tiles_with_a_rest", "one_row_tile", "two_row_tiles", "tokens_in_a_row"]


@pytest.mark.parametrize("bad", [-1, 0, 1 << 30], ids=["negative", "pages", "far"])
@pytest.mark.parametrize("kernel", KERNELS, ids=IDS)
def test_entries_outside_the_pool_read_as_zeros(sca, kernel, bad):
    dt, algo, group, T, lengths = kernel
    make = lambda: Setup(3, 2, group, T, 64, 16, lengths, None, DT[dt], seed=T, spare=0)
    s = make()
    table = s.table.clone()
    wrong = [1, 17, lengths[1] // 16]       # of request 1: in the first tile, further on, the newest rows'
    for e in wrong:
        table[1, e] = bad if bad else s.pages
    plan = lambda: sca.PagedTreeAttention(s.cache(sca), 3, s.H, tokens=T, keys=s.table.shape[1] * 16, algo=code_of(sca, algo))
    p, ok = plan(), plan()
    args = (s.q.cuda(), ints(lengths).cuda())
    o, lse = p.attend(args[0], table.cuda(), args[1])
    assert sca.capi.sca_read_status(p.status.data_ptr(), 0) == sca.capi.SCA_ERR_RANGE
    o2, lse2 = ok.attend(args[0], s.table.cuda(), args[1])
    assert ok.read_status() == 0
    assert torch.equal(o[[0, 2]], o2[[0, 2]]) and torch.equal(lse[[0, 2]], lse2[[0, 2]])
    z = make()
    for e in wrong:
        z.k[s.table[1, e].long()], z.v[s.table[1, e].long()] = 0, 0
    compare(o, lse, z, None, p.scale, dt == "bf16")


@pytest.mark.parametrize("kernel", KERNELS, ids=IDS)
def test_a_table_that_ends_before_the_rows(sca, kernel):
    """Rows behind it are not seen: the same as fewer rows, and reported."""
    dt, algo, group, T, lengths = kernel
    s = Setup(3, 2, group, T, 64, 16, lengths, None, DT[dt], seed=T, spare=0)
    n = 35                                   # entries: 560 rows
    cap = 16 * n
    plan = sca.PagedTreeAttention(s.cache(sca), 3, s.H, tokens=T, keys=cap, algo=code_of(sca, algo))
    short = s.table[:, :n].contiguous().cuda()
    o, lse = plan.attend(s.q.cuda(), short, ints(lengths).cuda())
    assert sca.capi.sca_read_status(plan.status.data_ptr(), 0) == sca.capi.SCA_ERR_RANGE
    for b in range(3):
        ref, rl, mag = as_far_as(s, b, cap, plan.scale)
        g, gl = o[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
        # tolerances as in compare (tests/test_gpu_paged.py); |q| and |k| below 14
        es = 64 * 2.0 ** -23 * 14 * 14 * plan.scale + 2.0 ** -21
        err = 2 * es + cap * 2.0 ** -23 + 2.0 ** -20 + (2.0 ** -8 if dt == "bf16" else 0.0)
        assert (np.abs(g - ref) <= HALF[s.dtype] * 1.01 * np.abs(ref) + err * mag).all(), b
        assert (np.abs(gl - rl) <= es + cap * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * np.abs(rl)).all(), b


def as_far_as(s, b, cap, scale):
    """The oracle's (o, lse, mean |v|) of request b, token by token over those of its rows that lie before `cap`."""
    parts = []
    for t in range(s.T):
        rows = min(s.lengths[b] + t + 1, cap)      # the last of them counts as the token's own
        parts.append(oracle.tree_attention(s.q[b:b + 1, :, t:t + 1], s.k, s.v, s.table[b:b + 1], [rows - 1], [1], None, scale))
    return tuple(np.concatenate([p[i][0] for p in parts], 1) for i in range(3))


@pytest.mark.parametrize("kernel", KERNELS, ids=IDS)
def test_heads_beyond_32_bits(sca, kernel):
    """Heads that lie 2^31 elements apart and more, pages 2^20: as in a pool of their own."""
    dt, algo, group, T, _ = kernel
    Hkv, D, page, pages, dtype = 2, 64, 16, 40, DT[dt]
    far = (1 << 31) + 4096
    pools, own = [], []
    for i in range(2):
        base = torch.empty(far + (1 << 20) * pages, dtype=dtype, device="cuda")
        x = torch.randn(pages, Hkv, page, D, generator=torch.Generator().manual_seed(i)).to(dtype).cuda()
        pools.append(base.as_strided((pages, Hkv, page, D), (1 << 20, far, D, 1)).copy_(x))
        own.append(x)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32)[None].cuda()
    lengths = ints([pages * page - T - 3]).cuda()
    q = torch.randn(1, Hkv * group, T, D, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    outs = []
    for ps in (pools, own):
        cache = sca.PagedKVCache(pages, Hkv, D, page=page, dtype=dtype, pools=tuple(ps))
        plan = sca.PagedTreeAttention(cache, 1, Hkv * group, tokens=T, keys=pages * page, algo=code_of(sca, algo))
        o, lse = plan.attend(q, table, lengths)
        assert plan.read_status() == 0 and torch.isfinite(o).all()
        outs.append((o.clone(), lse.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
