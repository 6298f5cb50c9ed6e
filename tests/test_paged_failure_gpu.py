"""Failure detection of paged attention without a GPU fault (as test_gpu_failure does for the linear):
the warps of products wait on a barrier that nothing arrives at, with a 1 ms limit. The kernels record
TTQ_ERR_TIMEOUT, drain the copies they started (all of them under way by then where a block has fewer
tiles than its ring has places) and leave no plan, since its counts of finished pieces are incomplete;
a new plan gives the results of before."""

import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq
from test_paged_gpu import Case

pytestmark = pytest.mark.gpu

TIMEOUT, INVALID = -6, -1


@pytest.mark.parametrize("new,length,max_new", [
    ([1, 1, 1], [40, 17, 130], 1),            # shares of a tile or two: the ring is never full
    ([1, 2], [40000, 9000], 2),               # split tiles, many turns of the ring
    ([20, 5], [64, 100], None), ([30, 200], [9000, 300], None), ([600], [7000], None)])
@pytest.mark.parametrize("D,opts", [(64, {}), (128, {}), (128, dict(softcap=20.0))])
def test_a_wait_that_runs_out(new, length, max_new, D, opts):
    c = Case(new, length, 8, 2, D, 64, seed=sum(length))
    plan = c.plan(max_new)
    attend = lambda out: ttq.paged_attention(c.qd, plan, c.kd, c.vd, c.td, out=out, **opts)
    good = attend(torch.zeros(c.N, 8 * D, dtype=torch.bfloat16, device="cuda"))
    assert ttq.device_status() == 0
    out = torch.full_like(good, 7.0)
    try:
        ttq.set_wait_limit_ns(1_000_000)
        ttq.debug_inject_stall(True)
        attend(out)
        status = ttq.device_status()
    finally:
        ttq.debug_inject_stall(False)
        ttq.set_wait_limit_ns(0)              # back to the default limit
    assert status == TIMEOUT
    assert ttq.device_status() == 0           # reading the status cleared it
    out.fill_(7.0)
    attend(out)                               # the next layer on that plan: no work, and a report
    assert ttq.device_status() == INVALID
    assert torch.all(out == 7.0)
    plan.update(c.start, c.ld)
    for _ in range(2):
        out.zero_()
        attend(out)
        assert ttq.device_status() == 0
        assert torch.equal(out, good)
