"""The decoder over a paged cache: its operators run together, as they are used. A prompt, its
branches and their steps against the dense decoder on the same weights and tokens (same TTQ
linears; the attentions differ by their roundings, so bars of the dense stack's tests), page
upkeep bit for bit, and scores against softmax in 64 bits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq
from online_activation_aware_b200 import synthetic
from online_activation_aware_b200.decoder import TTQDecoder
from online_activation_aware_b200.paged import PagedCache, PagedTTQDecoder

pytestmark = pytest.mark.gpu

SHAPE = dict(layers=2, heads=8, kv_heads=2, hidden=256, head_dim=128, inter=512)
# two attentions of the same inputs differ by at most their bars (8e-3 each), 4 TTQ linears a
# layer pass differences on and add codes' roundings (5e-3 each): 2 layers x (16e-3 + 20e-3)
STACK_RTOL = 7.2e-2


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


def build(cls, seed=5, r=0, **kw):
    w = synthetic.device_decoder_weights(SHAPE, r, seed)
    fn = torch.ones(SHAPE["hidden"], dtype=torch.bfloat16, device="cuda")
    return cls(SHAPE, w, fn, 4, 64, 0.5, 0.4, r=r, **kw)


def tokens(n, seed):
    return synthetic.as_bf16(synthetic.draw_hidden(n, SHAPE["hidden"], seed)).cuda()


@pytest.mark.parametrize("page_size,r", [(16, 0), (64, 16)])
def test_prefill_and_decode_follow_the_dense_decoder(page_size, r):
    T, steps = 150, 4
    dense = build(TTQDecoder, r=r, max_len=T + steps)
    paged = build(PagedTTQDecoder, r=r, max_len=T + steps, pages=24, page_size=page_size, max_seqs=2)
    x = tokens(T + steps, 3)
    assert rel(paged.prefill(x[:T]), dense.prefill(x[:T])) <= STACK_RTOL
    for i in range(steps):
        assert rel(paged.decode(x[T + i: T + i + 1]), dense.decode(x[T + i: T + i + 1])) <= STACK_RTOL
    assert paged.cache.length(paged.prompt) == T + steps
    assert ttq.device_status() == 0


def test_branches_follow_their_own_tokens():
    # three branches of one prompt (its last page half full, so each branch copies it), different
    # tokens, steps of one and of several tokens; each equals the same tokens on a sequence alone
    T = 41
    dec = build(PagedTTQDecoder, max_len=128, pages=40, page_size=16, max_seqs=8)
    x = tokens(T, 3)
    dec.prefill(x)
    a, b, c = dec.fork(count=3)
    free = dec.cache.free_pages
    new = [tokens(9, 10 + i) for i in range(3)]
    outs = [[], [], []]
    for lo, n in ((0, 1), (1, 1), (2, 5), (7, 2)):
        counts = [n, n, n]
        h = dec.step([a, b, c], torch.cat([t[lo: lo + n] for t in new]), counts)
        for i, part in enumerate(h.split(counts)):
            outs[i].append(part.clone())
    assert dec.cache.free_pages == free - 3 * (-(-(T + 9) // 16) - T // 16)
    assert len({tuple(dec.cache.page_list(s)[:2]) for s in (a, b, c, dec.prompt)}) == 1   # whole pages stay shared
    assert len({dec.cache.page_list(s)[2] for s in (a, b, c, dec.prompt)}) == 4           # the last one does not
    for i in range(3):
        alone = build(PagedTTQDecoder, max_len=128, pages=16, page_size=64, max_seqs=2)
        alone.prefill(x)
        want = torch.cat([alone.decode(new[i][j: j + 1]) for j in range(9)])
        assert rel(torch.cat(outs[i]), want) <= STACK_RTOL
    assert rel(torch.cat(outs[0]), torch.cat(outs[1])) > 0.3                              # and not each other
    for s in (a, b, c):
        dec.free(s)
    assert dec.cache.free_pages == free
    assert ttq.device_status() == 0


def test_ragged_step_equals_separate_steps():
    dec = build(PagedTTQDecoder, max_len=256, pages=40, page_size=32, max_seqs=8)
    dec.prefill(tokens(70, 3))
    s = dec.fork(count=4)
    t = tokens(60, 4)
    counts = [1, 40, 7, 12]
    h = dec.step([s[0], s[1], s[2], s[3]], t, counts)
    for i, part in enumerate(h.split(counts)):
        f = dec.fork()[0]
        want = dec.step([f], t[sum(counts[:i]): sum(counts[:i + 1])], [counts[i]])
        assert rel(part, want) <= STACK_RTOL
        dec.free(f)
    assert ttq.device_status() == 0


def test_compaction_leaves_the_answers():
    dec = build(PagedTTQDecoder, max_len=256, pages=40, page_size=16, max_seqs=8)
    dec.prefill(tokens(100, 3))
    a, b, c = dec.fork(count=3)
    t = tokens(60, 4)
    for s in (a, b, c):
        dec.step([s], t[:40], [40])
    dec.free(a)
    dec.cache.truncate(c, 120)
    before = {s: (dec.cache.length(s), [dec.cache.k[:, p].clone() for p in dec.cache.page_list(s)],
                  [dec.cache.v[:, p].clone() for p in dec.cache.page_list(s)]) for s in (b, c, dec.prompt)}
    free = dec.cache.free_pages
    assert dec.cache.compact() > 0 and dec.cache.compact() == 0
    assert dec.cache.free_pages == free
    held = {p for s in dec.cache.sequences for p in dec.cache.page_list(s)}
    assert max(held) == len(held) - 1
    for s, (n, ks, vs) in before.items():
        assert dec.cache.length(s) == n
        for p, k, v in zip(dec.cache.page_list(s), ks, vs):
            # (unwritten rows of a page may hold anything, NaN included: compare the bits)
            assert torch.equal(dec.cache.k[:, p].view(torch.int16), k.view(torch.int16))
            assert torch.equal(dec.cache.v[:, p].view(torch.int16), v.view(torch.int16))
        row = dec.cache.table[s].cpu().tolist()
        assert row[: len(ks)] == dec.cache.page_list(s)
    f = dec.fork(b)[0]
    want = dec.step([f], t[40:43], [3])
    assert rel(dec.step([b], t[40:43], [3]), want) <= 1e-6
    assert ttq.device_status() == 0


def test_scores_of_a_prompt_and_of_steps():
    V, T = 1000, 60
    head = synthetic.as_bf16(np.random.default_rng(9).normal(size=(V, SHAPE["hidden"])) / 16).cuda()
    dec = build(PagedTTQDecoder, max_len=128, pages=16, page_size=16, max_seqs=4, lm_head=head)
    h = dec.prefill(tokens(T, 3))
    tok = torch.randint(0, V, (T,), device="cuda")
    got = dec.score(h, tok, top=5, prefill=True)
    logits = dec.lm_head.decode(h).double()          # the head's own codes
    lp = torch.log_softmax(logits, -1)
    ref = lp[torch.arange(T), tok]
    # prefill and decode of a TTQ linear differ by their accumulation order only (bf16 logits of size
    # up to 8 then differ by a step of 2^-5 at most, and the sums by as much)
    assert (got["logprob"].double() - ref).abs().max() <= 2 * 2.0 ** -5
    assert (got["entropy"].double() + (lp.exp() * lp).sum(-1)).abs().max() <= 2 * 2.0 ** -5
    seqs = dec.fork(count=3)
    hs = dec.step(seqs, tokens(3, 4))
    one = dec.score(hs, torch.tensor([1, -1, 7], device="cuda"), top=3)
    logits = dec.lm_head.decode(hs)
    assert torch.equal(one["top_logprobs"].argsort(descending=True, stable=True), torch.arange(3, device="cuda").expand(3, 3))
    ref = torch.log_softmax(logits.double(), -1)
    assert abs(float(one["logprob"][0] - ref[0, 1])) <= 1e-4 and float(one["logprob"][1]) == 0.0
    assert torch.equal(one["top_ids"][:, 0], logits.float().argmax(-1))
    assert ttq.device_status() == 0


def test_cache_refusals_leave_it_as_it_was():
    c = PagedCache(1, 4, 16, 1, 64, max_seqs=2, max_len=64)
    a = c.new()
    c.extend([a], [40])
    c.fork(a)
    with pytest.raises(RuntimeError):
        c.fork(a)                                      # both sequences are in use
    state = (c.free_pages, c.sequences, [c.page_list(s) for s in c.sequences])
    with pytest.raises(ValueError):
        c.extend([a], [25])
    with pytest.raises(ValueError):
        c.extend([a, a], [1, 1])
    with pytest.raises(ValueError):
        c.extend([a], [0])
    with pytest.raises(KeyError):
        c.extend([7], [1])
    with pytest.raises(KeyError):
        c.free(9)
    with pytest.raises(ValueError):
        c.truncate(a, 41)
    assert (c.free_pages, c.sequences, [c.page_list(s) for s in c.sequences]) == state
    b = [s for s in c.sequences if s != a][0]
    with pytest.raises(RuntimeError):
        c.extend([a, b], [20, 20])                     # three pages and a copy, one page free
    assert (c.free_pages, c.sequences, [c.page_list(s) for s in c.sequences]) == state
    c.extend([b], [8])
    assert c.page_list(a)[:2] == c.page_list(b)[:2] and c.page_list(a)[2] != c.page_list(b)[2]


def test_branches_of_a_shared_last_page_take_what_is_there():
    # three holders of a half full page step at once: two copies, the third keeps it; two pages are free
    c = PagedCache(1, 5, 16, 1, 64, max_seqs=4, max_len=64)
    a = c.new()
    c.extend([a], [40])
    b, d = c.fork(a), c.fork(a)
    start, length, table = c.extend([a, b, d], [1, 2, 3])
    assert c.free_pages == 0
    assert sorted(c.page_list(s)[2] for s in (a, b, d)) == [2, 3, 4]
    assert start.tolist() == [0, 1, 3, 6] and length.tolist() == [41, 42, 43]
    assert [row[:3] for row in table.tolist()] == [c.page_list(s) for s in (a, b, d)]


def test_steps_of_many_sizes_share_one_scratch_buffer():
    dec = build(PagedTTQDecoder, max_len=256, pages=40, page_size=16, max_seqs=4)
    dec.prefill(tokens(100, 3))
    t = tokens(40, 4)
    sizes = []
    for n in (1, 33, 7):
        f = dec.fork()[0]
        dec.step([f], t[:n], [n])
        dec.free(f)
        sizes.append(dec.workspace(n).data_ptr())
    assert len(set(sizes)) == 1 and not dec._ws
    assert ttq.device_status() == 0


def test_decoder_refusals():
    dec = build(PagedTTQDecoder, max_len=64, pages=8, page_size=16, max_seqs=2)
    x = tokens(10, 3)
    with pytest.raises(RuntimeError):
        dec.step([0], x[:1])
    with pytest.raises(RuntimeError):
        dec.fork()
    dec.prefill(x)
    with pytest.raises(ValueError):
        dec.step([dec.prompt], x[:2])
    with pytest.raises(KeyError):
        dec.step([1], x[:1])
    with pytest.raises(RuntimeError):
        dec.score(x, torch.zeros(10, dtype=torch.int64, device="cuda"))
    with pytest.raises(NotImplementedError):
        dec.capture_decode()
    with pytest.raises(ValueError):
        dec.prefill(tokens(65, 3))
