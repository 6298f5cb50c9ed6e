"""Bookkeeping of the paged cache on the host (its tensors on the CPU, the page kernels replaced): a
call that fails on the way leaves the cache as it was."""

import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq
from online_activation_aware_b200.paged import PagedCache


def cache(**kw):
    return PagedCache(**{**dict(layers=2, pages=9, page_size=16, kv_heads=1, head_dim=64, max_seqs=4, max_len=64,
                                device="cpu"), **kw})


def state(c):
    return (c.free_pages, c.sequences, [c.page_list(s) for s in c.sequences], [c.length(s) for s in c.sequences],
            list(c._held), [c.table[s, : len(c.page_list(s))].tolist() for s in c.sequences])


def copied(k, v, src, dst):
    for t in (k, v):
        t[:, dst.long()] = t[:, src.long()].clone()


def remapped(table, mapping, out):
    out.copy_(torch.where(table >= 0, mapping[table.clamp(min=0).long()], table))


def fails(*args, **kw):
    raise torch.OutOfMemoryError("no memory")


@pytest.fixture
def kernels(monkeypatch):
    monkeypatch.setattr(ttq, "copy_pages", copied)
    monkeypatch.setattr(ttq, "remap_pages", remapped)
    return monkeypatch


def test_an_extension_that_fails_leaves_the_cache_as_it_was(kernels):
    c = cache()
    a = c.new()
    c.extend([a], [24])
    b, d = c.fork(a), c.fork(a)
    before = state(c)
    kernels.setattr(ttq, "copy_pages", fails)
    with pytest.raises(torch.OutOfMemoryError):
        c.extend([a, b, d], [9, 1, 30])
    assert state(c) == before
    kernels.setattr(ttq, "copy_pages", copied)
    kernels.setattr(c, "_upload", fails)
    with pytest.raises(torch.OutOfMemoryError):
        c.extend([b], [20])
    assert state(c) == before
    kernels.undo()
    kernels.setattr(ttq, "copy_pages", copied)
    start, length, table = c.extend([a, b, d], [9, 1, 30])
    assert start.tolist() == [0, 9, 10, 40] and length.tolist() == [33, 25, 54]
    assert [row[: len(c.page_list(s))] for row, s in zip(table.tolist(), (a, b, d))] == [c.page_list(s) for s in (a, b, d)]
    assert len({c.page_list(s)[0] for s in (a, b, d)}) == 1 and len({c.page_list(s)[1] for s in (a, b, d)}) == 3
    assert c.free_pages == 9 - 1 - 3 - 1 - 2 and sorted(c._held)[-1] == 3 and sum(c._held) == 3 + 2 + 4


@pytest.mark.parametrize("broken", ["copy_pages", "remap_pages"])
def test_a_compaction_that_fails_leaves_the_cache_as_it_was(kernels, broken):
    c = cache()
    a, b = c.new(), c.new()
    c.extend([a], [40])
    c.extend([b], [50])
    c.k.copy_(torch.randn_like(c.k, dtype=torch.float32).bfloat16())
    held = c.k[:, c.page_list(b)].clone()
    c.free(a)
    before = state(c)
    kernels.setattr(ttq, broken, fails)
    with pytest.raises(torch.OutOfMemoryError):
        c.compact()
    assert state(c) == before and torch.equal(c.k[:, c.page_list(b)], held)
    kernels.undo()
    kernels.setattr(ttq, "copy_pages", copied)
    kernels.setattr(ttq, "remap_pages", remapped)
    assert c.compact() == 3 and c.compact() == 0
    assert sorted(c.page_list(b)) == [0, 1, 2, 3] and torch.equal(c.k[:, c.page_list(b)], held)
    assert c.table[b, :4].tolist() == c.page_list(b) and c.free_pages == 5
