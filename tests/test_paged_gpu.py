"""Parity of the paged-cache operators with the fp64 oracle, on the same bf16 inputs.

Bars (a rounding is off by at most half a step: bf16 2^-8 of the value):
  attention   the kernels may round the softmax weights to bf16 for the tensor cores, in the
      numerator and the sum alike: a weight is off by at most 2 * 2^-8 of itself, the result
      then by 2^-7 sum w |v|, plus 2^-8 of itself for its own rounding, plus 1e-3 sum w |v| for
      fp32 scores (a score of size 20 summed over 128 products is off by less than
      128 * 2^-24 * 20, its capped form by as much again, and each weight by that fraction);
  q and k of the page write   as in test_decoder_gpu: one bf16 step of the fp64 value;
  log probabilities   fp32: the sums of up to 2^18 positive terms in chains of at most 2^10
      and a tree are off by less than 1e-4 of themselves in the worst case and 1e-5 in
      practice; the log of the sum by as much, the differences x - m are exact to 2^-24 |x - m|.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq
from online_activation_aware_b200 import synthetic
from oracle import paged_oracle as PO
from test_decoder_gpu import assert_ulp

pytestmark = pytest.mark.gpu

INVALID = -1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ttq.load_library()
    yield
    assert ttq.device_status() == 0


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def vals(t):
    return synthetic.bf16_values(t.cpu().contiguous())


class Case:
    """Sequences with `new` tokens over `length` positions; pages scattered over a pool whose
    unused parts hold NaN."""

    def __init__(self, new, length, H, Hkv, D, page, seed=0, pad=3, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.new, self.length, self.H, self.Hkv, self.D, self.page = list(new), list(length), H, Hkv, D, page
        need = [-(-L // page) for L in length]
        pool = sum(need) + 3
        order = rng.permutation(pool)
        self.table = np.full((len(new), max(max(need), 1)), -1, dtype=np.int64)
        k = torch.full((pool, page, Hkv, D), float("nan"))
        v = torch.full((pool, page, Hkv, D), float("nan"))
        at = 0
        for b, L in enumerate(length):
            self.table[b, :need[b]] = order[at: at + need[b]]
            at += need[b]
            p = torch.arange(L)
            row = torch.from_numpy(self.table[b])[p // page]
            k[row, p % page] = torch.randn(L, Hkv, D, generator=g) * scale
            v[row, p % page] = torch.randn(L, Hkv, D, generator=g) * torch.exp(0.5 * torch.randn(1, Hkv, D, generator=g))
        self.k, self.v = k.bfloat16(), v.bfloat16()
        self.N = sum(new) + pad
        self.pad = pad
        self.q = (torch.randn(self.N, H * D, generator=g) * scale).bfloat16()
        self.start = i32(np.concatenate([[0], np.cumsum(new)]))
        self.kd, self.vd, self.qd = self.k.cuda(), self.v.cuda(), self.q.cuda()
        self.td, self.ld = i32(self.table), i32(length)

    def want(self, **kw):
        return PO.attention(vals(self.q).reshape(self.N, self.H, self.D), vals(self.k), vals(self.v), self.table,
                            self.new, self.length, **kw)

    def plan(self, max_new=None, window=0, prefix=None):
        p = ttq.AttentionPlan(len(self.new), self.N, self.H, self.Hkv, self.D, max_new=max_new)
        return p.update(self.start, self.ld, window=window, prefix=None if prefix is None else i32(prefix))


def assert_attention(got, want, mag):
    n = want.shape[0]
    got = vals(got[:n]).reshape(want.shape)
    assert np.isfinite(got).all()
    tol = (2.0 ** -7 + 1e-3) * mag + 2.0 ** -8 * np.abs(want) + 1e-30
    worst = (np.abs(got - want) / tol).max() if n else 0.0
    assert worst <= 1.0, worst


def check(c, softcap=0.0, slopes=None, window=0, prefix=None, max_new=None):
    out = torch.full((c.N, c.H * c.D), 7.0, dtype=torch.bfloat16, device="cuda")
    sd = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
    plan = c.plan(max_new, window, prefix)
    ttq.paged_attention(c.qd, plan, c.kd, c.vd, c.td, softcap=softcap, slopes=sd, out=out)
    assert ttq.device_status() == 0
    assert_attention(out, *c.want(softcap=softcap, slopes=slopes, window=window, prefix=prefix))
    assert torch.all(out[c.N - c.pad:] == 7.0)          # rows behind the last sequence
    return out


# ------------------------------------------------------------------ attention


@pytest.mark.parametrize("H,Hkv,D,page", [(8, 8, 64, 16), (8, 4, 128, 32), (6, 2, 64, 64), (16, 4, 128, 16),
                                          (10, 2, 128, 128), (16, 2, 64, 256), (16, 1, 128, 64), (7, 1, 64, 32),
                                          (24, 1, 128, 32), (64, 1, 64, 16)])
def test_single_tokens(H, Hkv, D, page):
    length = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 700, 1023, 2500]
    check(Case([1] * len(length), length, H, Hkv, D, page, seed=H + D), max_new=1)


@pytest.mark.parametrize("H,Hkv,D,page", [(4, 4, 64, 16), (8, 4, 128, 64), (6, 2, 128, 32), (8, 2, 128, 16),
                                          (10, 2, 128, 64), (8, 1, 64, 128), (24, 1, 64, 32), (64, 1, 128, 256)])
def test_chunks(H, Hkv, D, page):
    new = [1, 7, 0, 130, 33, 64, 200, 1]
    length = [1, 7, 5, 130, 300, 65, 1111, 64]
    check(Case(new, length, H, Hkv, D, page, seed=H + D + page))


@pytest.mark.parametrize("new", [2, 3, 4, 5, 15, 16, 17])
def test_few_tokens_per_sequence(new):
    length = [new, new + 1, 64, 500, 1300]
    check(Case([new] * 5, length, 8, 2, 128, 32, seed=new), max_new=new)
    check(Case([new] * 5, length, 8, 2, 128, 32, seed=new))       # no bound given: any sequence may be long


@pytest.mark.parametrize("new,length,H,Hkv,D,opts", [
    ([30], [9000], 4, 1, 64, {}), ([20, 5], [7001, 300], 8, 2, 128, {}), ([17], [30000], 2, 1, 128, {}),
    ([200], [6000], 3, 1, 64, dict(window=3000, prefix=[500])), ([1, 90, 2], [5000, 4100, 2], 6, 1, 128, dict(softcap=20.0)),
    ([1], [40000], 2, 1, 64, {}), ([2, 1], [2600, 9000], 16, 2, 128, dict(window=2000))])
def test_few_tiles_over_a_long_context(new, length, H, Hkv, D, opts):
    # tiles in many pieces, several of them joined by one block; a plan used again by the next layer
    c = Case(new, length, H, Hkv, D, 64, seed=sum(length))
    bound = max(new)
    first = check(c, max_new=bound, **opts)
    plan = c.plan(bound, opts.get("window", 0), opts.get("prefix"))
    for _ in range(3):
        again = ttq.paged_attention(c.qd, plan, c.kd, c.vd, c.td, softcap=opts.get("softcap", 0.0))
        assert torch.equal(again[: sum(new)], first[: sum(new)])


def test_rows_that_see_nothing():
    # empty caches, and more new tokens than positions: the first of them lie before the start
    c = Case([1, 3, 5, 40], [0, 0, 2, 17], 8, 2, 64, 16)
    out = check(c)
    assert torch.all(out[:4] == 0) and torch.all(out[4:7] == 0) and torch.all(out[9:9 + 23] == 0)
    c = Case([1, 1, 1], [0, 1, 0], 8, 2, 128, 16)
    out = check(c, max_new=1)
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0)


def test_empty_step_leaves_everything():
    check(Case([0, 0], [10, 0], 8, 2, 64, 16, pad=4))
    check(Case([0, 0], [10, 0], 8, 2, 64, 16, pad=4), max_new=1)


@pytest.mark.parametrize("new,max_new", [([1, 1, 1, 1, 1], 1), ([1, 70, 200, 3, 129], None)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("opts", [dict(softcap=30.0), dict(softcap=2.0), dict(window=1), dict(window=64), dict(window=100),
                                  dict(prefix=[5, 0, 300, 64, 2000]), dict(window=33, prefix=[5, 0, 300, 64, 1]),
                                  dict(slopes=True), dict(softcap=20.0, slopes=True, window=90, prefix=[1, 2, 3, 130, 0])])
def test_masks_and_biases(opts, D, new, max_new):
    length = [3, 500, 1000, 300, 700]
    o = dict(opts)
    if o.get("slopes"):
        o["slopes"] = [2.0 ** (-1 - h) for h in range(8)]
    check(Case(new, length, 8, 2, D, 16, seed=11, scale=1.5), max_new=max_new, **o)


def test_distance_bias_over_a_long_context():
    # the sharp slopes leave the nearest positions only, the flat ones reach far back
    check(Case([1, 1], [20000, 16385], 8, 1, 64, 64, seed=5), max_new=1, slopes=[2.0 ** -(h + 1) for h in range(8)])


@pytest.mark.parametrize("max_new", [1, None])
def test_pages_outside_the_window_may_be_gone(max_new):
    # a sliding window's user frees old pages: their table entries and contents are not read
    c = Case([1, 1, 1], [800, 517, 96], 8, 2, 128, 16, seed=3)
    w = 40
    keep = [-(-(L - w + 1) // 16) * 16 - 16 for L in c.length]
    for b, L in enumerate(c.length):
        first = (L - w) // 16
        gone = c.table[b, :first].copy()
        c.td[b, :first] = -1
        c.kd[torch.from_numpy(gone)] = float("nan")
        c.vd[torch.from_numpy(gone)] = float("nan")
        # positions ahead of the window in the same page
        c.kd[c.table[b, first], : (L - w) % 16] = float("nan")
        c.vd[c.table[b, first], : (L - w) % 16] = float("inf")
    out = torch.empty(c.N, 8 * 128, dtype=torch.bfloat16, device="cuda")
    ttq.paged_attention(c.qd, c.plan(max_new, window=w), c.kd, c.vd, c.td, out=out)
    assert ttq.device_status() == 0
    assert_attention(out, *c.want(window=w))
    assert min(keep) >= 0


def test_large_scores_and_equal_scores():
    c = Case([1, 20], [300, 90], 8, 2, 128, 16, scale=6.0)     # scores up to hundreds: one weight takes all
    out = torch.empty(c.N, 8 * 128, dtype=torch.bfloat16, device="cuda")
    ttq.paged_attention(c.qd, c.plan(), c.kd, c.vd, c.td, out=out)
    want, mag = c.want()
    got = vals(out[:21]).reshape(want.shape)
    # a score of 400 in fp32 is off by up to 128 * 2^-24 * 400 = 3e-3
    assert (np.abs(got - want) <= (2.0 ** -7 + 8e-3) * mag + 2.0 ** -8 * np.abs(want)).all()
    c = Case([1, 20], [300, 90], 8, 2, 128, 16)
    c.qd.zero_()
    c.q.zero_()
    check(c)


def test_strided_queries_and_shared_pages():
    # q heads read in place from a stacked projection; two sequences on the same pages
    c = Case([1, 1, 30], [200, 200, 333], 8, 2, 128, 32, seed=9)
    c.table[1] = c.table[0]
    c.td = i32(c.table)
    wide = torch.full((c.N, 12 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, : 8 * 128] = c.qd
    out = ttq.paged_attention(wide, c.plan(), c.kd, c.vd, c.td)
    assert_attention(out, *c.want())
    assert ttq.device_status() == 0


@pytest.mark.parametrize("softcap", [1e-3, 1e6, 3e38])
@pytest.mark.parametrize("max_new", [1, None])
def test_extreme_caps(softcap, max_new):
    # a cap that flattens every score, and caps too large to matter
    check(Case([1, 1] if max_new else [1, 40], [200, 90], 8, 2, 128, 16, seed=4), max_new=max_new, softcap=softcap)


@pytest.mark.parametrize("softcap", [4.0, 7.0, 12.0, 24.0, 100.0])
@pytest.mark.parametrize("slopes", [None, [2.0 ** -i for i in range(8)]])
def test_caps_around_the_scores(softcap, slopes):
    # scores up to about 5: beyond the cap, inside it and far inside it, within one tile too
    c = Case([130, 3, 64], [700, 200, 64], 8, 2, 128, 32, seed=int(softcap))
    check(c, softcap=softcap, slopes=slopes)


def test_padding_rows_and_neighbours_do_not_leak():
    # NaN in the padding rows of q and in another sequence's own cache stays where it is
    c = Case([3, 20, 1], [40, 300, 17], 8, 2, 128, 16, seed=12, pad=5)
    c.qd[24:] = float("nan")
    c.kd[c.table[0][0]] = float("nan")
    c.vd[c.table[0][0]] = float("inf")
    out = torch.full((c.N, 8 * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ttq.paged_attention(c.qd, c.plan(), c.kd, c.vd, c.td, out=out)
    want, mag = c.want()
    assert_attention(out[3:24], want[3:], mag[3:])
    assert torch.all(out[24:] == 7.0) and ttq.device_status() == 0


def test_lists_at_any_alignment_and_a_wide_single_row():
    c = Case([1], [77], 8, 2, 64, 16, pad=0, seed=13)
    off = lambda t: torch.cat([t.new_zeros(3), t.reshape(-1)])[3:].view(t.shape)
    wide = torch.zeros(1, 8 * 64 + 5, dtype=torch.bfloat16, device="cuda")
    wide[:, : 8 * 64] = c.qd
    p = ttq.AttentionPlan(1, 1, 8, 2, 64).update(off(c.start), off(c.ld), prefix=off(i32([4])))
    out = ttq.paged_attention(wide, p, c.kd, c.vd, off(c.td), slopes=off(torch.full((8,), 0.1, device="cuda")))
    assert_attention(out, *c.want(prefix=[4], slopes=[0.1] * 8))
    assert ttq.device_status() == 0


def test_calls_on_another_stream():
    c = Case([1, 40], [300, 90], 8, 2, 128, 16, seed=14)
    side = torch.cuda.Stream()
    plan = ttq.AttentionPlan(2, c.N, 8, 2, 128)
    side.wait_stream(torch.cuda.current_stream())
    plan.update(c.start, c.ld, stream=side)
    out = ttq.paged_attention(c.qd, plan, c.kd, c.vd, c.td, stream=side)
    x = torch.randn(5, 9000, device="cuda")
    tok = torch.arange(5, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    got = ttq.token_logprobs(x, tok, 3, stream=side)
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]   # reuses freed memory, if any
    side.synchronize()
    assert_attention(out, *c.want())
    want = ttq.token_logprobs(x, tok, 3)
    assert all(torch.equal(got[k], want[k]) for k in want) and len(junk) == 8
    assert ttq.device_status() == 0


def test_results_repeat_bit_for_bit():
    c = Case([1, 5, 64, 1], [3000, 900, 4000, 17], 8, 2, 128, 64, seed=21)
    first = check(c)
    plan = c.plan()
    for _ in range(3):
        assert torch.equal(ttq.paged_attention(c.qd, plan, c.kd, c.vd, c.td)[: sum(c.new)], first[: sum(c.new)])


@pytest.mark.parametrize("new,max_new", [([1, 1, 1], 1), ([20, 150, 1], None)])
def test_captured_step_follows_new_lengths(new, max_new):
    c = Case(new, [900, 300, 64], 8, 2, 128, 16, seed=2)
    plans = [ttq.AttentionPlan(3, c.N, 8, 2, 128, max_new=max_new) for _ in range(2)]
    outs = [torch.zeros(c.N, 8 * 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lens = c.ld.clone()
    for p, o in zip(plans, outs):
        p.update(c.start, lens)
        ttq.paged_attention(c.qd, p, c.kd, c.vd, c.td, out=o)
    torch.cuda.synchronize()
    graphs = []
    for p, o in zip(plans, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.update(c.start, lens)
            ttq.paged_attention(c.qd, p, c.kd, c.vd, c.td, out=o)
            ttq.paged_attention(c.qd, p, c.kd, c.vd, c.td, out=o)   # a second layer on the same plan
        graphs.append(g)
    for length in ([900, 300, 64], [150, 250, 3], [870, 151, 40]):
        lens.copy_(i32(length))
        c.length = length
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        want = c.want()
        for o in outs:
            assert_attention(o, *want)
    assert ttq.device_status() == 0


def test_bad_lengths_and_pages_are_reported():
    c = Case([1, 2], [40, 30], 8, 2, 64, 16)
    out = torch.empty(c.N, 8 * 64, dtype=torch.bfloat16, device="cuda")
    for start, lens in (([0, 1, 9], [40, 30]), ([1, 1, 3], [40, 30]), ([0, 2, 1], [40, 30]), ([0, 1, 3], [40, -1])):
        p = ttq.AttentionPlan(2, c.N, 8, 2, 64)
        p.update(i32(start), i32(lens))
        assert ttq.device_status() == INVALID
        ttq.paged_attention(c.qd, p, c.kd, c.vd, c.td, out=out)     # an invalid plan: no work
        assert ttq.device_status() == INVALID
    # a plan of other sizes
    p = ttq.AttentionPlan(2, c.N, 8, 2, 64).update(c.start, c.ld)
    p.max_new = 5
    ttq.paged_attention(c.qd, p, c.kd, c.vd, c.td, out=out)
    assert ttq.device_status() == INVALID
    # lengths past the table, and entries that are no pages
    for max_new in (2, None):
        c.plan(max_new)
        p = ttq.AttentionPlan(2, c.N, 8, 2, 64, max_new=max_new).update(c.start, i32([40, 4000]))
        ttq.paged_attention(c.qd, p, c.kd, c.vd, c.td, out=out)
        assert ttq.device_status() == INVALID
        for bad in (-1, c.kd.shape[0], 2 ** 31 - 1):
            t = c.td.clone()
            t[1, 0] = bad
            ttq.paged_attention(c.qd, c.plan(max_new), c.kd, c.vd, t, out=out)
            assert ttq.device_status() == INVALID
    check(c)


# ------------------------------------------------------------------ page writes


@pytest.mark.parametrize("H,Hkv,D,page,new,length", [
    (8, 2, 128, 16, [1] * 40, list(range(1, 41))), (4, 4, 64, 32, [5, 0, 70, 1], [5, 3, 100, 33]),
    (6, 2, 256, 64, [33, 1], [200, 1]), (40, 8, 128, 16, [129, 64], [129, 1000]), (5, 1, 64, 16, [1], [500])])
def test_page_write(H, Hkv, D, page, new, length):
    c = Case(new, length, H, Hkv, D, page, seed=H + D)
    rng = np.random.default_rng(3)
    S = H + 2 * Hkv
    qkv = synthetic.as_bf16(rng.normal(size=(c.N, S * D)) * rng.lognormal(size=(1, S * D))).cuda()
    wq, wk = (synthetic.as_bf16(1 + 0.1 * rng.normal(size=D)).cuda() for _ in range(2))
    rope = ttq.rope_table(max(length), D, 1.0e6)
    kd, vd = c.kd.clone(), c.vd.clone()
    before = qkv.clone()
    q = torch.full((c.N, H * D), 7.0, dtype=torch.bfloat16, device="cuda")
    ttq.qk_norm_rope_paged(qkv, H, Hkv, D, wq, wk, 1e-6, rope, c.start, c.ld, kd, vd, c.td, q=q)
    assert ttq.device_status() == 0
    assert torch.equal(qkv, before) and torch.all(q[sum(new):] == 7.0)
    want_q, writes = PO.append(vals(qkv), H, Hkv, D, vals(wq), vals(wk), new, length, c.table, page)
    floor = 2.0 ** -20 * 2.0
    assert_ulp(q[: sum(new)].reshape(-1, H, D), want_q, floor)
    pages, slots = torch.tensor([w[0] for w in writes]), torch.tensor([w[1] for w in writes])
    assert_ulp(kd[pages, slots], np.array([w[2] for w in writes]), floor)
    np.testing.assert_array_equal(vals(vd[pages, slots]), np.array([w[3] for w in writes]))
    # everything else as it was (NaN included)
    kd[pages, slots] = c.kd[pages, slots]
    vd[pages, slots] = c.vd[pages, slots]
    assert torch.equal(kd.view(torch.int16), c.kd.view(torch.int16))
    assert torch.equal(vd.view(torch.int16), c.vd.view(torch.int16))


def test_page_write_gives_the_dense_cache():
    T, H, Hkv, D = 77, 8, 2, 128
    rng = np.random.default_rng(8)
    qkv = synthetic.as_bf16(rng.normal(size=(T, (H + 2 * Hkv) * D))).cuda()
    wq, wk = (synthetic.as_bf16(1 + 0.1 * rng.normal(size=D)).cuda() for _ in range(2))
    rope = ttq.rope_table(100, D, 1.0e6)
    kc, vc = (torch.zeros(96, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp, vp = (torch.zeros(6, 16, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = ttq.qk_norm_rope_paged(qkv, H, Hkv, D, wq, wk, 1e-6, rope, i32([0, T]), i32([T + 9]), kp, vp,
                               i32([[3, 1, 5, 0, 2, 4]]))
    dense = qkv.clone()
    ttq.qk_norm_rope(dense, H, Hkv, D, wq, wk, 1e-6, rope, 9, kc, vc)
    # the two kernels add a head's 128 squares in different orders, so their fp32 results differ by up
    # to 128 * 2^-24 of themselves and may round to neighbouring bf16 values, no further
    assert_ulp(q, vals(dense[:, : H * D]), 2.0 ** -19)
    order = torch.tensor([3, 1, 5, 0, 2, 4])
    assert_ulp(kp[order].reshape(96, Hkv, D)[: T + 9], vals(kc[: T + 9]), 2.0 ** -19)
    assert torch.equal(vp[order].reshape(96, Hkv, D)[: T + 9], vc[: T + 9])


def test_page_write_out_of_range_writes_nothing():
    c = Case([2, 1], [40, 20], 8, 2, 64, 16)
    qkv = torch.ones(c.N, 12 * 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    rope = ttq.rope_table(64, 64, 1.0e6)
    for start, lens, table in ((c.start, i32([40, 200]), c.td), (c.start, i32([40, 65]), c.td.expand(2, -1).contiguous()),
                               (c.start, i32([40, 0]), c.td), (i32([0, 2, 99]), c.ld, c.td),
                               (c.start, c.ld, torch.full_like(c.td, 99))):
        kd, vd = c.kd.clone(), c.vd.clone()
        ttq.qk_norm_rope_paged(qkv, 8, 2, 64, w, w, 1e-6, rope, start, lens, kd, vd, table)
        assert ttq.device_status() == INVALID
        if table is not c.td:
            continue
        # sequence 1's pages (and the unused ones) are untouched
        keep = torch.from_numpy(np.setdiff1d(np.arange(kd.shape[0]), c.table[0][c.table[0] >= 0]))
        if start is c.start:
            assert torch.equal(kd[keep].view(torch.int16), c.kd[keep].view(torch.int16))


# ------------------------------------------------------------------ pages


@pytest.mark.parametrize("layers,pages,page,Hkv,D,moves,dtype", [
    (1, 2, 16, 1, 64, 1, torch.bfloat16), (5, 40, 16, 2, 64, 20, torch.bfloat16), (3, 33, 7, 1, 24, 9, torch.float32),
    (36, 12, 32, 8, 128, 5, torch.bfloat16), (2, 9, 1, 1, 16, 4, torch.uint8), (1, 300, 64, 4, 128, 150, torch.bfloat16)])
def test_copy_pages(layers, pages, page, Hkv, D, moves, dtype):
    g = torch.Generator(device="cuda").manual_seed(moves)
    k, v = (torch.randint(0, 256, (layers, pages, page, Hkv, D * dtype.itemsize), generator=g, dtype=torch.uint8,
                          device="cuda").view(dtype) for _ in range(2))
    order = torch.randperm(pages, generator=g, device="cuda").int()
    src, dst = order[:moves].clone(), order[moves: 2 * moves].clone()
    src[moves // 2:] = src[0].clone()                       # several copies of one page
    wk, wv = k.clone().view(torch.uint8), v.clone().view(torch.uint8)
    for w in (wk, wv):
        w[:, dst.long()] = w[:, src.long()]
    ttq.copy_pages(k, v, src, dst)
    assert torch.equal(k.view(torch.uint8), wk) and torch.equal(v.view(torch.uint8), wv)
    # one layer given alone; a page onto itself
    k1 = k[layers - 1].clone()
    v1 = v[layers - 1].clone()
    ttq.copy_pages(k1, v1, src[:1], src[:1])
    assert torch.equal(k1.view(torch.uint8), wk[layers - 1])
    assert ttq.device_status() == 0


def test_copy_pages_out_of_range_is_skipped():
    k, v = (torch.arange(4 * 16, device="cuda", dtype=torch.float32).view(1, 4, 1, 1, 16).contiguous() for _ in range(2))
    v = v + 100
    before = k.clone()
    ttq.copy_pages(k, v, i32([0, 4, -1]), i32([1, 2, 3]))
    assert ttq.device_status() == INVALID
    assert torch.equal(k[0, 1], before[0, 0]) and torch.equal(k[0, 2:], before[0, 2:])
    ttq.copy_pages(k, v, i32([0, 0]), i32([4, -1]))
    assert ttq.device_status() == INVALID
    ttq.copy_pages(k, v, i32([]), i32([]))


def test_remap_pages():
    rng = np.random.default_rng(0)
    for shape in ((1, 1), (3, 300), (257, 13)):
        t = i32(rng.integers(-1, 50, size=shape))
        m = i32(rng.permutation(50))
        want = torch.where(t < 0, t, m[t.clamp(min=0).long()])
        assert torch.equal(ttq.remap_pages(t, m), want)
        assert torch.equal(ttq.remap_pages(t, m, out=t), want) and torch.equal(t, want)
    out = ttq.remap_pages(i32([0, 50, 1]), torch.full((50,), 50, dtype=torch.int32, device="cuda"))
    assert out.tolist() == [-1, -1, -1]
    assert ttq.device_status() == INVALID


# ------------------------------------------------------------------ log probabilities


def check_logprobs(x, tokens, top):
    got = ttq.token_logprobs(x, tokens, top)
    x64 = x.float().cpu().numpy().astype(np.float64)
    lp, ent, ids, tlp = PO.logprobs(x64, tokens.cpu().numpy(), top)
    span = np.nanmax(np.where(np.isfinite(x64), np.abs(x64), 0)) + 1

    def near(a, b):
        # sums off by 1e-5 of themselves; x - m and the logarithm rounded at their size
        np.testing.assert_allclose(a.cpu().numpy(), b, rtol=2e-6, atol=2e-5 + span * 2.0 ** -23)

    near(got["logprob"], lp)
    near(got["entropy"], ent)
    if top:
        np.testing.assert_array_equal(got["top_ids"].cpu().numpy(), ids)
        near(got["top_logprobs"], tlp)
    else:
        assert set(got) == {"logprob", "entropy"}
    assert ttq.device_status() == 0
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (1, 5, 5), (3, 7, 0), (2, 1000, 20), (5, 4097, 32), (1, 50257, 20),
                                            (150, 2049, 1), (33, 131072, 5), (2, 200001, 32), (400, 333, 32)])
def test_token_logprobs(rows, vocab, top, dtype):
    g = torch.Generator(device="cuda").manual_seed(vocab + rows)
    x = (3 * torch.randn(rows, vocab, generator=g, device="cuda")).to(dtype)
    tok = torch.randint(-1, vocab, (rows,), generator=g, device="cuda")
    check_logprobs(x, tok, top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "spike", "banned", "huge", "two", "zeros"])
@pytest.mark.parametrize("rows,vocab", [(2, 33000), (200, 1500)])
def test_token_logprobs_orders_and_extremes(kind, dtype, rows, vocab):
    ramp = torch.arange(vocab, device="cuda", dtype=torch.float32).expand(rows, -1) / 100
    x = {"equal": torch.full((rows, vocab), 1.5, device="cuda"), "rising": ramp, "falling": -ramp,
         "spike": torch.zeros(rows, vocab, device="cuda"), "banned": torch.zeros(rows, vocab, device="cuda"),
         "huge": 3.0e37 * torch.sin(ramp), "two": torch.zeros(rows, vocab, device="cuda"),
         "zeros": torch.where(ramp.int() % 2 == 0, 0.0, -0.0)}[kind].clone()
    if kind == "spike":
        x[:, vocab - 1] = 80.0
    if kind == "banned":
        x[:, ::3] = -float("inf")
        x[0, :] = -float("inf")
        x[0, 1] = 2.0
    if kind == "two":
        x[:] = -30000.0
        x[:, 5] = 0.0
        x[:, vocab // 2] = 0.0
    tok = torch.arange(rows, device="cuda") * 7 % vocab
    tok[0] = 1
    check_logprobs(x.to(dtype), tok, 32)


def test_token_logprobs_of_rows_without_a_distribution():
    x = torch.randn(6, 5000, device="cuda")
    x[0, 77] = float("nan")
    x[1, 78] = float("inf")
    x[2] = -float("inf")
    x[3] = float("nan")
    x[4, 10:] = float("nan")
    tok = torch.tensor([0, 1, 2, 3, 4, 5], device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        got = check_logprobs(x.to(dtype), tok, 20)
        assert torch.isnan(got["logprob"][:5]).all() and torch.isnan(got["entropy"][:5]).all()
        assert torch.isfinite(got["logprob"][5])


def test_token_logprobs_strided_rows_and_bad_tokens():
    wide = torch.full((9, 1033), float("nan"), device="cuda")
    wide[:, :1001] = torch.randn(9, 1001, device="cuda")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        check_logprobs(wide.to(dtype)[:, :1001], torch.arange(9, device="cuda"), 10)
    for dtype in (torch.float32, torch.bfloat16):           # rows and columns of a larger tensor
        check_logprobs(torch.randn(9, 5001, device="cuda").to(dtype)[3:, 7:], torch.arange(6, device="cuda"), 10)
    x = torch.randn(3, 100, device="cuda")
    got = ttq.token_logprobs(x, torch.tensor([100, 1, 2 ** 40], device="cuda"))
    assert torch.isnan(got["logprob"][[0, 2]]).all() and torch.isfinite(got["logprob"][1])
    assert ttq.device_status() == INVALID


def test_token_logprobs_captured():
    x = torch.randn(4, 40000, device="cuda")
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    ttq.token_logprobs(x, tok, 5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ttq.token_logprobs(x, tok, 5)
    for s in range(3):
        x.copy_(torch.randn(4, 40000, device="cuda"))
        tok.fill_(s)
        g.replay()
        want = check_logprobs(x, tok, 5)
        for name in want:
            assert torch.equal(got[name], want[name])


# ---------------------------------------------------------------- arguments


def test_tensors_of_the_wrong_kind_are_refused():
    H, Hkv, D, B, W, page = 8, 2, 64, 2, 3, 16
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    i = lambda *s: z(*s, dt=torch.int32)
    plan = ttq.AttentionPlan(B, 4, H, Hkv, D, max_new=3)
    qs, kl, pt = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda"), i(B) + 20, i(B, W)
    k, v = z(4, page, Hkv, D), z(4, page, Hkv, D)
    q = z(4, H * D)
    plan.update(qs, kl)
    att = lambda **o: ttq.paged_attention(**{**dict(q=q, plan=plan, k_pages=k, v_pages=v, page_table=pt), **o})
    for wrong, kind in ((dict(q=q.half()), TypeError), (dict(q=q.cpu()), ValueError), (dict(q=z(3, H * D)), ValueError),
                        (dict(q=z(4, H * D - 8)), ValueError), (dict(q=z(H * D, 4).t()), ValueError),
                        (dict(k_pages=k.float()), TypeError), (dict(v_pages=z(5, page, Hkv, D)), ValueError),
                        (dict(k_pages=z(4, page, D, Hkv).transpose(2, 3)), ValueError),
                        (dict(page_table=pt.long()), TypeError), (dict(page_table=i(B + 1, W)), ValueError),
                        (dict(page_table=i(W, B).t()), ValueError), (dict(slopes=z(H)), TypeError),
                        (dict(slopes=z(H + 1, dt=torch.float32)), ValueError), (dict(out=z(4, H * D + 8)), ValueError),
                        (dict(softcap=-1.0), ttq.TTQError), (dict(softcap="a"), TypeError), (dict(q=None), TypeError),
                        (dict(k_pages=z(4, 24, Hkv, D), v_pages=z(4, 24, Hkv, D)), ttq.TTQError)):
        with pytest.raises(kind):
            att(**wrong)
    for wrong, kind in ((dict(q_start=qs[:2]), ValueError), (dict(q_start=qs.long()), TypeError),
                        (dict(kv_len=kl.cpu()), ValueError), (dict(prefix=i(B + 1)), ValueError),
                        (dict(window=-1), ttq.TTQError), (dict(window=1.5), TypeError)):
        with pytest.raises(kind):
            plan.update(**{**dict(q_start=qs, kv_len=kl), **wrong})
    with pytest.raises(ttq.TTQError):
        ttq.token_logprobs(z(2, 10), torch.zeros(2, dtype=torch.int64, device="cuda"), top=11)
    with pytest.raises(ttq.TTQError):
        ttq.token_logprobs(z(2, 10), torch.zeros(2, dtype=torch.int64, device="cuda"), top=-1)
    out = z(4, H * D) + 3
    assert att(out=out) is out and torch.count_nonzero(out) == 0
    table = i(B, W)
    assert ttq.remap_pages(table, i(4) + 2, out=table) is table and bool((table == 2).all())
    assert ttq.device_status() == 0
