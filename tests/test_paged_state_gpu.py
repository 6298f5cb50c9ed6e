"""The paged decoder after calls that fail: a step or a prompt that is refused, or that fails in one of
its layers, leaves no positions that were never written, and no prompt that is half quantized."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq
from online_activation_aware_b200 import synthetic
from online_activation_aware_b200.paged import PagedTTQDecoder
from test_paged_decoder_gpu import SHAPE, build, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ttq.load_library()
    yield
    assert ttq.device_status() == 0


def make(**kw):
    return build(PagedTTQDecoder, **{**dict(max_len=128, pages=24, page_size=16, max_seqs=4), **kw})


def state(dec):
    c = dec.cache
    return c.free_pages, c.sequences, [c.page_list(s) for s in c.sequences], [c.length(s) for s in c.sequences]


def stop_at(layer):
    def trace(li, name, t):
        if li == layer and name == "attn":
            raise torch.OutOfMemoryError("no memory")
    return trace


def wrong_rows(n):
    """Rows that a step of n tokens has to refuse."""
    good = tokens(n, 4)
    return [(good.float(), TypeError), (good.cpu(), ValueError), (good[:, :-8].contiguous(), ValueError),
            (good[0] if n == 1 else good.view(-1), ValueError)]


def test_a_failed_step_leaves_the_sequences():
    x, new = tokens(41, 3), tokens(3, 4)
    want = make()
    want.prefill(x)
    wf = want.fork()[0]
    w0, w1 = want.step([wf], new, [3]), want.step([want.prompt, wf], new[:2])
    dec = make()
    dec.prefill(x)
    f = dec.fork()[0]
    before = state(dec)
    for bad, kind in wrong_rows(3):
        with pytest.raises(kind):
            dec.step([f], bad, [3])
        assert state(dec) == before
    for layer in (0, 1):
        with pytest.raises(torch.OutOfMemoryError):
            dec.step([f, dec.prompt], tokens(30, 5), [20, 10], trace=stop_at(layer))
        after = state(dec)
        # lengths as before; a branch may keep its own copy of the last page
        assert after[1] == before[1] and after[3] == before[3]
        assert [len(p) for p in after[2]] == [len(p) for p in before[2]]
    with pytest.raises(torch.OutOfMemoryError):
        dec._plan, plan = (lambda *a: stop_at(0)(0, "attn", None)), dec._plan
        try:
            dec.step([f], new, [3])
        finally:
            dec._plan = plan
    assert state(dec)[3] == before[3]
    assert torch.equal(dec.step([f], new, [3]), w0)
    assert torch.equal(dec.step([dec.prompt, f], new[:2]), w1)


def test_a_failed_prompt_leaves_none():
    x, other, new = tokens(41, 3), tokens(20, 6), tokens(2, 4)
    dec = make()
    dec.prefill(x)
    before = state(dec)
    for bad, kind in wrong_rows(41) + [(x[:0], ValueError), (tokens(129, 3), ValueError)]:
        with pytest.raises(kind):
            dec.prefill(bad)
        assert state(dec) == before and dec.prompt is not None     # refused: the prompt before is still there
    want = make()
    want.prefill(x)
    assert torch.equal(dec.step([dec.prompt], new[:1]), want.step([want.prompt], new[:1]))
    with pytest.raises(torch.OutOfMemoryError):
        dec.prefill(other, trace=stop_at(1))
    assert dec.prompt is None and dec.cache.sequences == [] and dec.cache.free_pages == dec.cache.pages
    for call in (lambda: dec.step([0], new[:1]), lambda: dec.decode(new[:1]), dec.fork):
        with pytest.raises(RuntimeError):
            call()
    assert torch.equal(dec.prefill(x), make().prefill(x))


def test_the_head_answers_with_codes_of_this_prompt_only():
    head = synthetic.as_bf16(np.random.default_rng(9).normal(size=(1000, SHAPE["hidden"])) / 16).cuda()
    tok = torch.arange(30, device="cuda")
    dec = make(lm_head=head)
    h = dec.prefill(tokens(30, 3))
    with pytest.raises(RuntimeError):
        dec.score(h, tok)                                   # no codes at all
    first = dec.score(h, tok, top=3, prefill=True)
    again = dec.score(h, tok, top=3)
    assert (first["logprob"] - again["logprob"]).abs().max() <= 2 * 2.0 ** -5   # (bf16 logits of size up to 8)
    other = dec.prefill(tokens(30, 6))
    with pytest.raises(RuntimeError):
        dec.score(other, tok)                               # codes of the prompt before
    got = dec.score(other, tok, top=3, prefill=True)
    want = make(lm_head=head)
    want = want.score(want.prefill(tokens(30, 6)), tok, top=3, prefill=True)
    assert all(torch.equal(got[k], want[k]) for k in want)
    with pytest.raises(TypeError):
        dec.score(other.float(), tok, prefill=True)         # fails underway: the head has no codes
    with pytest.raises(RuntimeError):
        dec.score(other, tok)


@pytest.mark.parametrize("through_cache", [False, True])
def test_a_freed_prompt_is_not_mistaken_for_another_sequence(through_cache):
    new = tokens(2, 4)
    dec = make()
    dec.prefill(tokens(41, 3))
    a = dec.fork()[0]
    dec.step([a], new[:1])
    (dec.cache if through_cache else dec).free(dec.prompt)
    assert dec.prompt is None
    b = dec.fork(a)[0]                                      # takes the prompt's number
    assert b == 0 and dec.prompt is None
    before = state(dec)
    for call in (lambda: dec.decode(new[:1]), dec.fork):
        with pytest.raises(RuntimeError):
            call()
    assert state(dec) == before
    assert torch.equal(dec.step([a], new[1:]), dec.step([b], new[1:]))


def test_a_fork_of_more_than_there_is_room_for_makes_none():
    dec = make()                                            # four sequences
    dec.prefill(tokens(41, 3))
    before = state(dec)
    with pytest.raises(RuntimeError):
        dec.fork(count=4)
    with pytest.raises(KeyError):
        dec.fork(3, count=4)
    assert state(dec) == before
    assert dec.fork(count=0) == [] and dec.fork(count=3) == [1, 2, 3]


def test_rows_of_any_strides():
    x, new = tokens(41, 3), tokens(3, 4)
    want = make()
    wp = want.prefill(x)
    ws = want.step([want.prompt], new, [3])
    wide = lambda t: torch.cat([t, t], 1)[:, : t.shape[1]]
    across = lambda t: t.t().contiguous().t()
    for strided in (wide, across):
        dec = make()
        assert torch.equal(dec.prefill(strided(x)), wp)
        assert torch.equal(dec.step([dec.prompt], strided(new), [3]), ws)
