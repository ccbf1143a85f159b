"""A plan's first call on another stream than the one that it was made on, which
is busy, or captured: the counters in its workspace are zeros by then."""
import pytest
import torch

from tests.test_gpu_paged import Setup, attend, ints, sca  # noqa: F401

pytestmark = pytest.mark.gpu


def setup(T):
    return Setup(1, 1, 4, T, 64, 64, [9000], None, torch.bfloat16, seed=T)   # units in many pieces


@pytest.mark.parametrize("T", [1, 16])
def test_first_call_while_the_plan_is_still_being_zeroed(sca, T):
    s = setup(T)
    algo = sca.capi.SCA_ALGO_TC
    plan, o, lse = attend(sca, s, None, algo)
    want = (o.clone(), lse.clone())
    args = (s.q.cuda(), s.table.cuda(), ints(s.lengths).cuda())
    n = plan._ws.numel()
    pools = (plan.cache.k, plan.cache.v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.full((n,), 1, dtype=torch.int32, device="cuda")   # what the workspace's memory held
            torch.cuda._sleep(100_000_000)                          # about 50 ms
            cache = sca.PagedKVCache(s.pages, s.Hkv, s.D, page=s.page, pools=pools)
            late = sca.PagedTreeAttention(cache, s.B, s.H, tokens=T, keys=s.table.shape[1] * s.page, algo=algo)
        assert not side.query()
        o, lse = late.attend(*args)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and late.read_status() == 0
        assert not late._ws[:1024].any()


@pytest.mark.parametrize("inside", [False, True])
def test_first_call_in_a_capture(sca, inside):
    s = setup(16)
    algo = sca.capi.SCA_ALGO_TC
    plan, o, lse = attend(sca, s, None, algo)     # (loads the kernels)
    want = (o.clone(), lse.clone())
    args = (s.q.cuda(), s.table.cuda(), ints(s.lengths).cuda())
    make = lambda: sca.PagedTreeAttention(plan.cache, s.B, s.H, tokens=16, keys=s.table.shape[1] * s.page, algo=algo)
    made = None if inside else make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = made or make()
        o, lse = made.attend(*args)
    for _ in range(3):
        o.zero_()
        graph.replay()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and made.read_status() == 0
    if not inside:      # and as ordinary calls
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o, lse = made.attend(*args)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
