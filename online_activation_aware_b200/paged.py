"""Several sequences that share one prompt: a cache made of pages and a decoder over it.

TTQ's codes belong to a prompt: every layer is re-quantized from the prompt's own
activations. Branches of a prompt (parallel samples, beams, alternative turns) therefore
share its codes, and their decode steps run as rows of one TTQ linear. ``PagedCache`` gives
them a key/value cache of pages, shared until a branch writes to one, and
``PagedTTQDecoder`` is ``TTQDecoder`` over it: ``prefill`` a prompt, ``fork`` it, ``step``
any of its sequences by one or several tokens each, ``score`` the answer.
"""

from __future__ import annotations

import heapq

import torch

import online_activation_aware_b200 as ttq
from online_activation_aware_b200.decoder import TTQDecoder


class PagedCache:
    """Key/value pools [layers, pages, page_size, kv_heads, head_dim] (bf16) and the pages of up
    to ``max_seqs`` sequences of up to ``max_len`` positions.

    The bookkeeping (free pages, how many sequences hold each page) lives on the host; the page
    tables live on the device (``table`` [max_seqs, width] int32) and follow it. Pages that
    several sequences hold are never written: ``extend`` gives a sequence its own copy of a
    shared last page first. Every call acts on the current stream; one that raises leaves the
    cache as it was."""

    def __init__(self, layers: int, pages: int, page_size: int, kv_heads: int, head_dim: int, max_seqs: int,
                 max_len: int, device="cuda"):
        if pages < 1 or max_seqs < 1 or max_len < 1:
            raise ValueError("pages, max_seqs and max_len must be positive")
        self.pages, self.page_size, self.max_seqs, self.max_len = pages, page_size, max_seqs, max_len
        self.width = -(-max_len // page_size)
        self.k = torch.empty(layers, pages, page_size, kv_heads, head_dim, dtype=torch.bfloat16, device=device)
        self.v = torch.empty_like(self.k)
        self.table = torch.full((max_seqs, self.width), -1, dtype=torch.int32, device=device)
        self._births = 0
        self.clear()

    def clear(self):
        """Forgets every sequence."""
        self._free = list(range(self.pages))       # a heap: the lowest page first
        self._held = [0] * self.pages              # sequences that hold each page
        self._pages = {}                           # sequence -> its pages
        self._length = {}
        self._born = {}                            # which of all sequences that ever had the number

    @property
    def free_pages(self) -> int:
        return len(self._free)

    @property
    def sequences(self) -> list:
        return sorted(self._pages)

    def length(self, seq: int) -> int:
        self._check(seq)
        return self._length[seq]

    def page_list(self, seq: int) -> list:
        """The pages of a sequence, in order."""
        self._check(seq)
        return list(self._pages[seq])

    def _check(self, seq):
        if seq not in self._pages:
            raise KeyError(f"no sequence {seq}")

    def new(self) -> int:
        """An empty sequence."""
        for seq in range(self.max_seqs):
            if seq not in self._pages:
                self._pages[seq], self._length[seq] = [], 0
                self._births += 1
                self._born[seq] = self._births
                return seq
        raise RuntimeError(f"all {self.max_seqs} sequences are in use")

    def fork(self, seq: int) -> int:
        """A new sequence with the same positions, sharing their pages."""
        self._check(seq)
        other = self.new()
        self._pages[other] = list(self._pages[seq])
        self._length[other] = self._length[seq]
        for p in self._pages[seq]:
            self._held[p] += 1
        self.table[other].copy_(self.table[seq])
        return other

    def free(self, seq: int):
        """Ends a sequence; pages that no other holds become free, and so does its number."""
        self._check(seq)
        for p in self._pages.pop(seq):
            self._release(p)
        del self._length[seq], self._born[seq]

    def truncate(self, seq: int, length: int):
        """Drops the positions from ``length`` on (rejected tokens), with pages left without any."""
        self._check(seq)
        if not 0 <= length <= self._length[seq]:
            raise ValueError(f"sequence {seq} has {self._length[seq]} positions")
        keep = -(-length // self.page_size)
        for p in self._pages[seq][keep:]:
            self._release(p)
        del self._pages[seq][keep:]
        self._length[seq] = length

    def _release(self, p):
        self._held[p] -= 1
        if self._held[p] == 0:
            heapq.heappush(self._free, p)

    def _upload(self, values):
        """One host list of int32 values on the device, behind the current stream's work."""
        return torch.tensor(values, dtype=torch.int32).to(self.table.device, non_blocking=True)

    def extend(self, seqs, counts):
        """Makes room for counts[i] more positions of sequence seqs[i]; shared pages that these
        reach are copied first. Returns the step's device tensors (q_start, kv_len, page_table)."""
        seqs, counts = list(seqs), list(counts)
        if len(seqs) == 0 or len(set(seqs)) != len(seqs) or len(seqs) != len(counts):
            raise ValueError("one count for each of at least one distinct sequences")
        need = 0
        left = {}   # holders of a shared last page, less those that copy it here
        copying = set()
        for s, n in zip(seqs, counts):
            self._check(s)
            if n < 1:
                raise ValueError("every sequence takes at least one token")
            if self._length[s] + n > self.max_len:
                raise ValueError(f"{self._length[s] + n} positions exceed {self.max_len}")
            held = len(self._pages[s])
            need += -(-(self._length[s] + n) // self.page_size) - held
            if self._length[s] % self.page_size:
                last = self._pages[s][-1]
                if left.setdefault(last, self._held[last]) > 1:
                    left[last] -= 1
                    need += 1
                    copying.add(s)
        if need > len(self._free):
            raise RuntimeError(f"{need} pages are needed, {len(self._free)} are free")
        src, dst, where, taken, own, added, lengths = [], [], [], [], {}, {}, {}

        def take():
            taken.append(heapq.heappop(self._free))
            return taken[-1]

        # the bookkeeping follows once the device's part is under way: a call that raises leaves it as it was
        try:
            for s, n in zip(seqs, counts):
                held, new = len(self._pages[s]), []
                if s in copying:
                    own[s] = take()
                    src.append(self._pages[s][-1])
                    dst.append(own[s])
                    where.append((s, held - 1, own[s]))
                lengths[s] = self._length[s] + n
                while (held + len(new)) * self.page_size < lengths[s]:
                    new.append(take())
                    where.append((s, held + len(new) - 1, new[-1]))
                added[s] = new
            # one upload: copies, table entries, the step's starts, lengths and rows (each part padded to
            # 16 bytes)
            starts = [0]
            for n in counts:
                starts.append(starts[-1] + n)
            parts = [src, dst, [s * self.width + i for s, i, _ in where], [p for _, _, p in where], starts,
                     [lengths[s] for s in seqs], seqs]
            flat, at = [], []
            for part in parts:
                at.append(len(flat))
                flat += part + [0] * (-len(part) % 4)
            up = self._upload(flat)
            src_d, dst_d, idx_d, new_d, start_d, len_d, row_d = (up[a: a + len(part)] for a, part in zip(at, parts))
            idx_d = idx_d.long()
            rows = torch.empty(len(seqs), self.width, dtype=torch.int32, device=self.table.device)
            if src:
                ttq.copy_pages(self.k, self.v, src_d, dst_d)
            if where:
                self.table.view(-1).index_copy_(0, idx_d, new_d)
            torch.index_select(self.table, 0, row_d, out=rows)
        except BaseException:
            for p in taken:
                heapq.heappush(self._free, p)
            raise
        for p in src:
            self._held[p] -= 1
        for p in taken:
            self._held[p] = 1
        for s, p in own.items():
            self._pages[s][-1] = p
        for s in seqs:
            self._pages[s] += added[s]
        self._length.update(lengths)
        return start_d, len_d, rows

    def compact(self) -> int:
        """Moves the held pages to the lowest places, so that the pools end in one run of free
        pages; returns how many moved."""
        held = [p for p in range(self.pages) if self._held[p]]
        holes = [p for p in range(len(held)) if not self._held[p]]
        movers = [p for p in held if p >= len(held)]
        if not movers:
            return 0
        mapping = list(range(self.pages))
        for p, h in zip(movers, holes):
            mapping[p] = h
        pad = -len(movers) % 4
        up = self._upload(movers + [0] * pad + holes + [0] * pad + mapping)
        n = len(movers) + pad
        ttq.copy_pages(self.k, self.v, up[: len(movers)], up[n: n + len(movers)])
        ttq.remap_pages(self.table, up[2 * n:], out=self.table)
        for p, h in zip(movers, holes):  # (last, as in extend)
            self._held[h], self._held[p] = self._held[p], 0
        for s in self._pages:
            self._pages[s] = [mapping[p] for p in self._pages[s]]
        self._free = list(range(len(held), self.pages))
        return len(movers)


class PagedTTQDecoder(TTQDecoder):
    """``TTQDecoder`` whose sequences share one prompt and live in a ``PagedCache``.

    ``prefill(x)`` starts a prompt (re-quantizing every layer; sequences of an earlier prompt
    end) and leaves its sequence in ``prompt``; ``fork`` branches a sequence; ``step`` runs new
    tokens of several sequences, one or more each, as the rows of one decode step with the
    prompt's codes. With ``lm_head`` (bf16 [vocab, hidden]) the output head is one more TTQ
    linear, and ``score`` gives log probabilities."""

    def __init__(self, shape: dict, weights: list, final_norm, q: int, g: int, alpha: float, lam: float, r: int = 0,
                 pages: int = 256, page_size: int = 64, max_seqs: int = 16, max_len: int = 4096 + 128, eps: float = 1e-6,
                 rope_base: float = 1.0e6, lm_head=None, device="cuda"):
        self._cache_args = (pages, page_size, max_seqs)
        super().__init__(shape, weights, final_norm, q, g, alpha, lam, r, max_len, eps, rope_base, device)
        self.lm_head = None if lm_head is None else ttq.TTQLinear(lm_head, q, g, alpha, lam)
        self._head_ready = False  # the head's codes are of this prompt

    def _make_cache(self):
        pages, page_size, max_seqs = self._cache_args
        self.cache = PagedCache(len(self.layers), pages, page_size, self.Hkv, self.D, max_seqs, self.max_len,
                                self.device)
        self._prompt = None   # (sequence, which of its number) once a prompt's codes are in the layers
        self._plans = {}
        self._needs, self._scratch = {}, None

    @property
    def prompt(self) -> int | None:
        """The prompt's own sequence; None before a prefill and once that sequence was freed (its
        branches go on, and its number may be another sequence's)."""
        if self._prompt is None or self.cache._born.get(self._prompt[0]) != self._prompt[1]:
            return None
        return self._prompt[0]

    def _own(self) -> int:
        if self._prompt is None:
            raise RuntimeError("a prefill comes first")
        if self.prompt is None:
            raise RuntimeError("the prompt's own sequence was freed")
        return self.prompt

    def workspace(self, T: int):
        """One scratch buffer for steps of any number of rows: it grows to the largest need."""
        if T not in self._needs:
            lins = [lin for L in self.layers for lin in L["lin"].values()]
            lins += [] if self.lm_head is None else [self.lm_head]
            self._needs[T] = max(ttq.workspace_size(T, lin.d, lin.d_out, lin.cfg) for lin in lins)
        if self._scratch is None or self._scratch.numel() < self._needs[T]:
            self._scratch = torch.empty(max(self._needs[T], 256), dtype=torch.uint8, device=self.device)
        return self._scratch

    def _attention(self, li: int, qkv, T: int, prefill: bool):
        start, length, pages, plan = self._step
        nm, k, v = self.layers[li]["norms"], self.cache.k[li], self.cache.v[li]
        q = ttq.qk_norm_rope_paged(qkv, self.H, self.Hkv, self.D, nm["n_q"], nm["n_k"], self.eps, self.table, start,
                                   length, k, v, pages)
        return q, ttq.paged_attention(q, plan, k, v, pages)

    def _plan(self, seqs: int, tokens: int, longest: int):
        key = (seqs, tokens, longest)
        if key not in self._plans:
            if len(self._plans) >= 16:
                self._plans.clear()
            self._plans[key] = ttq.AttentionPlan(seqs, tokens, self.H, self.Hkv, self.D, max_new=longest,
                                                 device=self.device)
        return self._plans[key]

    def _run_step(self, x, seqs, counts, prefill: bool, trace=None):
        before = [(s, self.cache.length(s)) for s in seqs]
        start, length, pages = self.cache.extend(seqs, counts)
        try:
            plan = self._plan(len(seqs), x.shape[0], max(counts)).update(start, length)
            self._step = (start, length, pages, plan)
            return self._stack(x, prefill, trace)
        except BaseException:
            for s, n in before:  # positions that some layer may not have written
                self.cache.truncate(s, n)
            raise
        finally:
            self._step = None

    def _check_rows(self, x):
        if x.dim() != 2 or x.shape[1] != self.hidden:
            raise ValueError(f"x must be [tokens, {self.hidden}], got {tuple(x.shape)}")
        if x.dtype != torch.bfloat16:
            raise TypeError(f"x must be bfloat16, got {x.dtype}")
        if x.device != self.cache.k.device:
            raise ValueError(f"x is on {x.device}, the cache on {self.cache.k.device}")

    def prefill(self, x, trace=None):
        """Embeddings [T, hidden] bf16 of a new prompt -> final-normed hidden [T, hidden]; its
        sequence is ``prompt``. Ends every sequence of the prompt before it (unless x is refused); when
        it fails underway there is no prompt."""
        self._check_rows(x)
        if x.shape[0] < 1:
            raise ValueError("a prompt has at least one token")
        if x.shape[0] > self.max_len:
            raise ValueError(f"{x.shape[0]} tokens exceed the cache of {self.max_len}")
        if -(-x.shape[0] // self.cache.page_size) > self.cache.pages:
            raise RuntimeError(f"{x.shape[0]} tokens exceed {self.cache.pages} pages of {self.cache.page_size}")
        self.cache.clear()
        self._head_ready = False
        seq = self.cache.new()
        self._prompt = (seq, self.cache._born[seq])
        try:
            return self._run_step(x, [seq], [x.shape[0]], True, trace)
        except BaseException:
            self.cache.clear()
            self._prompt = None  # the layers' codes may be of two prompts
            raise

    def step(self, seqs, x, counts=None, trace=None):
        """New tokens' embeddings x [sum counts, hidden], counts[i] (default one) of sequence
        seqs[i] -> their final-normed hidden states. A step that raises leaves the sequences at
        their length before it."""
        if self._prompt is None:
            raise RuntimeError("step needs a prefill first")
        self._check_rows(x)
        seqs = list(seqs)
        counts = [1] * len(seqs) if counts is None else list(counts)
        if sum(counts) != x.shape[0]:
            raise ValueError(f"{x.shape[0]} rows for {sum(counts)} tokens")
        return self._run_step(x, seqs, counts, False, trace)

    def decode(self, x, trace=None):
        """The next token of the prompt's own sequence."""
        return self.step([self._own()], x, None, trace)

    def capture_decode(self):
        raise NotImplementedError("steps of a paged decoder take their pages from the host")

    def fork(self, seq: int | None = None, count: int = 1) -> list:
        """``count`` new sequences that continue ``seq`` (default: the prompt's)."""
        if seq is None:
            seq = self._own()
        self.cache.length(seq)  # (there is such a sequence)
        left = self.cache.max_seqs - len(self.cache.sequences)
        if count > left:
            raise RuntimeError(f"{count} sequences are asked for, {left} of {self.cache.max_seqs} are free")
        return [self.cache.fork(seq) for _ in range(count)]

    def free(self, seq: int):
        self.cache.free(seq)

    def score(self, hidden, tokens, top: int = 0, prefill: bool = False):
        """Log probabilities of ``tokens`` (int64, one a row of the final-normed hidden states),
        entropies and the ``top`` alternatives, through the output head. ``prefill`` quantizes
        the head from these rows (a prompt's); later calls reuse its codes, until the next prompt."""
        if self.lm_head is None:
            raise RuntimeError("the decoder has no output head")
        if not prefill and not self._head_ready:
            raise RuntimeError("the output head has no codes of this prompt: score the prompt with prefill=True first")
        ws = self.workspace(hidden.shape[0])
        if prefill:
            self._head_ready = False
            logits = self.lm_head.prefill(hidden, ws=ws)
            self._head_ready = True
        else:
            logits = self.lm_head.decode(hidden, ws=ws)
        return ttq.token_logprobs(logits, tokens, top)
