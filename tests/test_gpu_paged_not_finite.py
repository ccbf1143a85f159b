"""Values that are not finite in a paged cache: padding and rows that see
nothing are 0 and -inf by every kernel, whatever the rows of the cache hold, and
an older row's value shows in the rows that see it, in its feature."""
import pytest
import torch

from tests.test_gpu_paged import DT, Setup, code_of, ints, sca  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [
    # kernel, dtype, algo, Hkv, group, D, older rows of request 0, spare pages
    ("few_fp32_rows", "f32", "auto", 2, 2, 64, 100, 2), ("few_fp32_rows_cut", "f32", "auto", 1, 2, 128, 6000, 2),
    ("fp32_tiles_cut", "f32", "auto", 2, 16, 64, 700, 2), ("fp32_tiles_cut", "f32", "auto", 2, 16, 128, 3000, 2),
    ("fp32_tiles_whole", "f32", "auto", 220, 16, 64, 100, 32), ("bf16_in_fp32", "bf16", "simt", 2, 2, 128, 300, 2),
    ("few_rows", "bf16", "tc", 2, 2, 64, 100, 2), ("few_rows_cut", "bf16", "tc", 1, 4, 128, 6000, 2),
    ("one_row_tile", "bf16", "tc", 2, 16, 64, 100, 2), ("one_row_tile_cut", "bf16", "tc", 1, 16, 128, 6000, 2),
    ("two_row_tiles_cut", "bf16", "tc", 1, 50, 64, 6000, 2),
]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[3]}x{c[4]}-{c[5]}")
def test_rows_that_see_nothing_stay_zero(sca, case, bad):
    """Request 0: two of four tokens are padding, an older row's value is not
    finite.  Request 1: no older rows, token 1 sees nothing, token 2's value is not
    finite.  Request 2: only padding."""
    _, dt, algo, Hkv, group, D, older, spare = case
    T, page, odd = 4, 16, 5                     # odd: the feature
    s = Setup(3, Hkv, group, T, D, page, [older, 0, 30], [2, 4, 0], DT[dt], seed=older + group, spare=spare)
    tree = torch.tensor([[0b1, 0b11, 0b101, 0b1001], [0b1, 0, 0b100, 0b1001], [0b1, 0b11, 0b101, 0b1001]],
                        dtype=torch.int64)
    plan = sca.PagedTreeAttention(s.cache(sca), 3, s.H, tokens=T, keys=s.table.shape[1] * page, algo=code_of(sca, algo))
    args = (s.q.cuda(), s.table.cuda(), ints(s.lengths).cuda())
    kw = dict(counts=ints(s.counts).cuda(), tree=tree.cuda())
    clean = tuple(t.clone() for t in plan.attend(*args, **kw))
    for b, row in ((0, older - 30), (1, 2)):
        plan.cache.v[int(s.table[b, row // page]), 0, row % page, odd] = bad
    plan.o.fill_(7.0)
    o, lse = plan.attend(*args, **kw)
    assert plan.read_status() == 0
    nothing = torch.zeros(3, T, dtype=torch.bool, device="cuda")
    nothing[0, 2:] = nothing[1, 1] = nothing[2] = True
    for x, l in (clean, (o, lse)):
        x = x.transpose(1, 2)
        assert not x[nothing].any() and torch.isneginf(l.transpose(1, 2)[nothing]).all()
    assert torch.equal(lse, clean[1])
    # the older row: in every live row of its head, in its feature alone
    assert not torch.isfinite(o[0, :group, :2, odd]).any()
    # (the newest token's value may show in any live row of its request and head, in its feature)
    free = torch.zeros_like(o, dtype=torch.bool)
    free[:2, :group, :, odd] = True
    assert torch.equal(o[~free], clean[0][~free])


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[3]}x{c[4]}-{c[5]}")
def test_an_infinite_key_stays_out_of_padding(sca, case):
    """Scores of +inf with an older row: NaN in the rows that see it, by the
    formula, and nothing in padding, whose queries the caller need not clear."""
    _, dt, algo, Hkv, group, D, older, spare = case
    T, page, odd = 4, 16, 5
    s = Setup(2, Hkv, group, T, D, page, [older, 300], [2, 1], DT[dt], seed=older + group + 1, spare=spare)
    s.q[..., odd] = s.q[..., odd].abs() + 0.5
    plan = sca.PagedTreeAttention(s.cache(sca), 2, s.H, tokens=T, keys=s.table.shape[1] * page, algo=code_of(sca, algo))
    args = (s.q.cuda(), s.table.cuda(), ints(s.lengths).cuda())
    kw = dict(counts=ints(s.counts).cuda())
    clean = tuple(t.clone() for t in plan.attend(*args, **kw))
    for b, row in ((0, 40), (1, 17)):
        plan.cache.k[int(s.table[b, row // page]), 0, row % page, odd] = float("inf")
    plan.o.fill_(7.0)
    o, lse = plan.attend(*args, **kw)
    assert plan.read_status() == 0
    hit = torch.zeros(2, s.H, T, dtype=torch.bool, device="cuda")
    hit[0, :group, :2] = hit[1, :group, :1] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])
