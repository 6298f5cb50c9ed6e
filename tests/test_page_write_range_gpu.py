"""The page write on values that are out of range: what it reports, and that every pool row is as a write
of the valid tokens alone leaves it. With few rows a group of lanes takes one head slot, with many (here
padding behind the last sequence) four."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq
from test_paged_gpu import Case, i32

pytestmark = pytest.mark.gpu

INVALID = -1
H, HKV, D, PAGE = 8, 2, 64, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ttq.load_library()
    yield
    assert ttq.device_status() == 0


class Write:
    def __init__(self, new, length, pad):
        self.c = Case(new, length, H, HKV, D, PAGE, pad=pad, seed=3)
        g = torch.Generator().manual_seed(1)
        self.qkv = torch.randn(self.c.N, (H + 2 * HKV) * D, generator=g).bfloat16().cuda()
        self.w = torch.ones(D, dtype=torch.bfloat16, device="cuda")

    def __call__(self, start, lens, table, rope_rows=64):
        kd, vd = self.c.kd.clone(), self.c.vd.clone()
        q = torch.full((self.c.N, H * D), 7.0, dtype=torch.bfloat16, device="cuda")
        ttq.qk_norm_rope_paged(self.qkv, H, HKV, D, self.w, self.w, 1e-6, ttq.rope_table(rope_rows, D, 1.0e6),
                               i32(start), i32(lens), kd, vd, table, q=q)
        return ttq.device_status(), kd.view(torch.int16), vd.view(torch.int16), q


@pytest.mark.parametrize("pad", [3, 13000])
@pytest.mark.parametrize("start,lens,table,rope_rows,valid", [
    ([0, 2, 3], [40, 200], None, 256, 2),           # past the page table
    ([0, 2, 3], [40, 65], "wide", 64, 2),           # past the rotary table, in pages that are there
    ([0, 2, 3], [40, 64], "wide", 64, 3),           # (its last row)
    ([0, 2, 3], [40, 0], None, 64, 2),              # ahead of the first position
    ([0, 2, 3], [1, 20], None, 64, -1),             # the first token ahead of it, the second not
    ([0, 2, 99999], [40, 20], None, 64, 2),         # more tokens than rows
    ([0, 2, 3], [40, 20], "none", 64, 0),           # entries that are no pages
    ([0, 2, -1], [40, 20], None, 64, 0),            # starts that decrease
    ([0, 3, 2], [40, 20], None, 64, 0),
    ([1, 2, 3], [40, 20], None, 64, 0)])
def test_only_valid_tokens_are_written(start, lens, table, rope_rows, valid, pad):
    w = Write([2, 1], [40, 20], pad)
    t = w.c.td
    if table == "none":
        t = torch.full_like(t, 99)
    if table == "wide":                             # sequence 1 reaches 128 positions of pages, its own and the unused
        rest = np.setdiff1d(np.arange(w.c.kd.shape[0]), w.c.table[0][w.c.table[0] >= 0])
        t = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
        t[0, :3] = w.c.td[0, :3]
        t[1] = i32(np.resize(rest, 8))
    status, k, v, q = w(start, lens, t, rope_rows)
    if valid == 3:
        assert status == 0
        last = int(t[1, 3])
        assert bool((k[last, 15] != w.c.kd.view(torch.int16)[last, 15]).any())
        return
    assert status == INVALID
    changed = (k != w.c.kd.view(torch.int16)).flatten(2).any(-1).nonzero().tolist()
    if valid == 0:
        assert changed == [] and torch.equal(v, w.c.vd.view(torch.int16)) and torch.all(q == 7.0)
    elif valid == 2:                                # sequence 0 as a write of it alone leaves the pools
        ok, wk, wv, wq = w([0, 2, 2], [40, 0], w.c.td, rope_rows)
        assert ok == 0
        assert torch.equal(k, wk) and torch.equal(v, wv) and torch.equal(q[:2], wq[:2])
    else:                                           # token 1 of sequence 0 and sequence 1's
        assert sorted(changed) == sorted([[int(t[0, 0]), 0], [int(t[1, 1]), 3]])
    assert torch.all(q[3:] == 7.0)                  # rows behind the last sequence
