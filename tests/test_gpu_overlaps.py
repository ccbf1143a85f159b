"""Views that lie between one another's rows: turned in place in one projection's
output, appended to pools whose pages hold keys and values, equal to tensors of
their own, bit for bit."""
import pytest
import torch

from tests.test_gpu_paged import DT, ints, sca  # noqa: F401

pytestmark = pytest.mark.gpu


def rnd(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_one_projection_turned_in_place(sca, dt, layout):
    capi = sca.capi
    B, H, Hkv, S, D = 3, 6, 2, 37, 64
    angles = sca.RotaryAngles(32, layout=layout)
    qkv = rnd(B, S, H + 2 * Hkv, D, seed=1, dtype=DT[dt])
    q, k, v = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
    q1, k1 = sca.RotaryPositions(B, H, S, D, angles, kv_heads=Hkv, dtype=DT[dt]).forward(q, k)
    before = v.clone()
    d = capi.sca_rotary_dims()
    d.B, d.H, d.Hkv, d.D, d.S, d.rotary_dim, d.amplitude = B, H, Hkv, D, S, 32, 1.0
    d.dtype, d.interleaved = capi.SCA_BF16 if dt == "bf16" else capi.SCA_F32, int(layout == "interleaved")
    d.q = d.qo = d.k = d.ko = capi.view(*q.stride()[:3])
    capi.rotary_apply(d, q.data_ptr(), k.data_ptr(), angles.turns.data_ptr(), None, q.data_ptr(), k.data_ptr(),
                      torch.cuda.current_stream().cuda_stream)
    assert torch.equal(q, q1) and torch.equal(k, k1) and torch.equal(v, before)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows_first", [False, True])
def test_pools_between_one_another_and_queries_in_place(sca, dt, rows_first):
    B, H, Hkv, T, D, page, pages = 2, 4, 2, 5, 64, 16, 9
    dtype, angles = DT[dt], sca.RotaryAngles(64)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:8].to(torch.int32).view(2, 4).cuda()
    lengths = ints([14, 31]).cuda()
    q, k, v = (rnd(B, h, T, D, seed=i, dtype=dtype) for i, h in enumerate((H, Hkv, Hkv)))

    def pools(both):
        one = [both[:, :, 0], both[:, :, 1]] if rows_first else [both[:, 0], both[:, 1]]
        return tuple(t.transpose(1, 2) if rows_first else t for t in one)

    shape = (pages, page, 2, Hkv, D) if rows_first else (pages, 2, Hkv, page, D)
    both = rnd(*shape, seed=9, dtype=dtype)
    own = sca.PagedKVCache(pages, Hkv, D, page=page, dtype=dtype, angles=angles,
                           pools=tuple(t.contiguous() for t in pools(both)))
    inner = sca.PagedKVCache(pages, Hkv, D, page=page, dtype=dtype, angles=angles, pools=pools(both))
    made = [sca.PagedTreeAttention(c, B, H, tokens=T, keys=64) for c in (own, inner)]
    want = made[0].append(q, k, v, table, lengths).clone()
    assert torch.equal(made[1].append(q, k, v, table, lengths), want)
    path, accepted = ints([[1, 3, 0, 0, 0], [0, 2, 4, 0, 0]]).cuda(), ints([2, 3]).cuda()
    assert all(p.accept(table, lengths, path, accepted).tolist() == [16, 34] for p in made)
    assert torch.equal(own.k, inner.k) and torch.equal(own.v, inner.v)
    # the C function over its own queries, half of a request padding
    capi, d = sca.capi, own.make_dims(B, T, 4, 4)
    d.H = H
    d.q, d.k, d.v = (capi.view(*t.stride()[:3]) for t in (q, k, v))
    counts, x = ints([5, 2]).cuda(), q.clone()
    capi.paged_kv_append(d, x.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(), lengths.data_ptr(),
                         counts.data_ptr(), None, angles.turns.data_ptr(), own.k.data_ptr(), own.v.data_ptr(),
                         x.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    want[1, :, 2:] = 0
    assert torch.equal(x, want)
    with pytest.raises(sca.ScaError):     # the plan's own queries as keys
        made[0].append(q, made[0].q[:, :Hkv], v, table, lengths)
    with pytest.raises(sca.ScaError):
        own.append(own.k.as_strided((B, Hkv, T, D), k.stride()), v, table, lengths)
    with pytest.raises(sca.ScaError):
        sca.PagedKVCache(pages, Hkv, D, page=page, dtype=dtype, pools=(own.k, own.k)).append(k, v, table, lengths)
    assert own.read_status() == 0 and inner.read_status() == 0
