"""A bounded wait of the linear's kernels that runs out while every copy of a CTA is already under way:
few enough K blocks that the ring of stages is never full, so the warp that starts the copies has
nothing to wait for. As in test_gpu_failure the kernel records TTQ_ERR_TIMEOUT, lets its copies land
and returns."""

import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq
from online_activation_aware_b200 import synthetic

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.mark.parametrize("T,d,d_out", [(256, 256, 512), (300, 128, 264), (24, 512, 256), (40, 128, 72),
                                       (256, 512, 512), (300, 512, 264)])  # (the last two on CTA pairs)
def test_a_wait_that_runs_out_behind_the_last_copy(T, d, d_out):
    X, W = synthetic.draw_layer(T, d, d_out, seed=5)
    Xb, Wb = synthetic.as_bf16(X).cuda(), synthetic.as_bf16(W).cuda()
    cfg = ttq.make_config(4, 64, 0.5, 0.4)
    good = ttq.linear_prefill(Xb, Wb, cfg)
    assert ttq.device_status() == 0
    again = lambda: ttq.linear_decode(Xb, good["s"], good["codes"], good["scale"], good["zero"], cfg, d_out)
    want = again()
    try:
        ttq.set_wait_limit_ns(1_000_000)
        ttq.debug_inject_stall(True)
        again()
        status = ttq.device_status()
    finally:
        ttq.debug_inject_stall(False)
        ttq.set_wait_limit_ns(0)  # back to the default limit
    assert status == TIMEOUT
    assert ttq.device_status() == 0
    assert torch.equal(again(), want) and ttq.device_status() == 0
