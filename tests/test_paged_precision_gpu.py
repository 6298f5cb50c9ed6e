"""Precision of paged attention beyond the bars of test_paged_gpu: what the softmax weights lose.

A sequence of few rows is held to the weights of the dense decode (fp32 there). Its kernel multiplies
the weights as a bf16 value and the bf16 of what that leaves: off by at most 2^-8 * 2^-8 = 2^-16 of
themselves. The scores here are products of one channel, exact in fp32 but for the scale to log2 units
and the exponential: |s| <= 4 is 6 in log2 units, off by 6 * 2^-23 and so 2^-20 of a weight, 2^-22 for the
hardware's power of two. Sums of at most 200 terms add 2^-17 at the worst. In all below 2^-15 of
sum w |v|, and half a bf16 step (2^-8 of the value) for the result.

In every kernel a row's numerator and sum take the same weights, so that equal values come out as
they went in: (sum w c) / (sum w) = c to fp32, which is c once rounded to bf16."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq
from test_paged_gpu import Case, vals

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ttq.load_library()
    yield
    assert ttq.device_status() == 0


def attend(c, max_new, **kw):
    out = ttq.paged_attention(c.qd, c.plan(max_new), c.kd, c.vd, c.td, **kw)
    assert ttq.device_status() == 0
    return out[: sum(c.new)]


@pytest.mark.parametrize("new,length,H,Hkv", [([1, 1, 1, 1], [3, 17, 64, 200], 8, 2), ([1, 1], [40, 130], 4, 4),
                                              ([2, 1, 4], [20, 90, 33], 8, 2), ([1, 1], [75, 16], 16, 1)])
def test_few_rows_weigh_values_like_the_dense_decode(new, length, H, Hkv):
    c = Case(new, length, H, Hkv, 64, 16, seed=H + sum(length), pad=0)
    g = torch.Generator().manual_seed(7)
    q, k = c.q.view(c.N, H, 64), c.k
    q[..., 1:] = 0
    k[..., 1:] = torch.where(torch.isnan(k[..., 1:]), k[..., 1:], torch.zeros_like(k[..., 1:]))
    q[..., 0] = (1 + torch.rand(c.N, H, generator=g)).bfloat16() * 4     # scores q k / 8
    k[..., 0] = torch.where(torch.isnan(k[..., 0]), k[..., 0], k[..., 0].clamp(-4, 4))
    # values of one size and either sign, so that weights of different keys cancel in many channels
    c.v.copy_(torch.where(torch.isnan(c.v), c.v, torch.sign(c.v)))
    c.qd, c.kd, c.vd = c.q.cuda(), c.k.cuda(), c.v.cuda()
    got = vals(attend(c, max(new)))
    want, mag = c.want()
    tol = 2.0 ** -15 * mag + 2.0 ** -8 * np.abs(want) + 1e-30
    worst = (np.abs(got.reshape(want.shape) - want) / tol).max()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("new,length,max_new", [([1, 1, 1], [5, 700, 3000], 1), ([1, 130, 300, 20], [9, 700, 2500, 4000], None)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("opts", [dict(), dict(softcap=30.0), dict(slopes=True)])
def test_equal_values_come_out_as_they_are(new, length, max_new, D, opts):
    # peaked scores: most of a row's weight is on one key, far above the maximum of the tiles before it
    c = Case(new, length, 8, 2, D, 16, seed=D + len(new), pad=0, scale=2.5)
    value = (1 + torch.arange(2 * D) % 7 / 8).bfloat16().view(2, D)
    c.vd = torch.where(torch.isnan(c.v), c.v, value.expand_as(c.v)).cuda()
    if opts.get("slopes"):
        opts = dict(slopes=torch.tensor([2.0 ** -(h + 4) for h in range(8)], device="cuda"))
    got = attend(c, max_new, **opts).view(-1, 2, 4, D)
    assert int((got != value.cuda().view(1, 2, 1, D)).sum()) == 0
