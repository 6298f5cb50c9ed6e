"""Cases of the serving operators: attention over a paged key/value cache, the write of new
keys and values into pages, the upkeep of pages, and token log probabilities.

``listed()`` gives fixed cases, ``draw()`` more of the same ranges. ``prepare`` makes what a
serving program has in hand before the call, ``run`` makes one pass: in elementary torch
operations (``own`` false) or through this repository's entry points (``own`` true).
``exact`` computes the same outputs in 64 bits from the definitions.
"""

import math
import random

import torch

own = False

BF16 = torch.bfloat16
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases


def _attention(name, seqs, new, length, heads, kv_heads, head_dim, page, lens_seed, softcap=0.0, slopes=False, window=0,
               prefix=0):
    """`seqs` sequences with new[0] .. new[1] new tokens each, over length[0] .. length[1]
    cached positions (the new ones included; sizes spread over their logarithm)."""
    return {"name": name, "op": "attention", "seqs": seqs, "new_lo": new[0], "new_hi": new[1], "len_lo": length[0],
            "len_hi": length[1], "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "lens_seed": lens_seed, "softcap": softcap, "slopes": slopes, "window": window, "prefix": prefix}


def _append(name, seqs, new, length, heads, kv_heads, head_dim, page, lens_seed):
    return {"name": name, "op": "append", "seqs": seqs, "new_lo": new[0], "new_hi": new[1], "len_lo": length[0],
            "len_hi": length[1], "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "lens_seed": lens_seed}


def _pages(name, layers, pages, moves, kv_heads, head_dim, page, rows, width):
    """`moves` pages of a pool of `pages` copied in every layer; with rows > 0 the page tables
    [rows, width] are rewritten for it."""
    return {"name": name, "op": "pages", "layers": layers, "pages": pages, "moves": moves, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "rows": rows, "width": width}


def _logprobs(name, rows, vocab, dtype, top):
    return {"name": name, "op": "logprobs", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top}


def listed():
    return [
        # the smallest step: one request, one new token, a short context (0.6B-shaped heads): latency
        _attention("decode-1x700", 1, (1, 1), (700, 700), 16, 8, 128, 16, 1),
        # a serving batch, one new token each, contexts of very unequal length (8B-shaped heads): bandwidth
        _attention("decode-64-ragged", 64, (1, 1), (300, 9000), 32, 8, 128, 32, 2),
        # few requests over long contexts (32B-shaped heads): the work is split along the context
        _attention("decode-3-long", 3, (1, 1), (60000, 131000), 64, 8, 128, 64, 3),
        # several follow-up turns of unequal length behind their caches (8B-shaped heads)
        _attention("turns-6", 6, (90, 700), (1000, 6000), 32, 8, 128, 32, 4),
        # one long chunk of a long prompt (14B-shaped heads, five query heads a key head): tensor bound
        _attention("chunk-4096", 1, (4096, 4096), (16411, 16411), 40, 8, 128, 64, 5),
        # turns and single tokens in one batch: capped scores, distance bias, window and a kept prefix
        _attention("mixed-masked", 24, (1, 300), (200, 9000), 12, 4, 64, 16, 6, 30.0, True, 1000, 70),
        # keys and values of one decode step into pages
        _append("append-64", 64, (1, 1), (300, 9000), 32, 8, 128, 32, 7),
        # keys and values of ragged prompts into pages
        _append("append-prompts", 9, (400, 1900), (500, 5000), 32, 8, 128, 32, 8),
        # branches forked from one prompt: each copies the shared last page, in every layer
        _pages("fork-7", 36, 64, 7, 8, 128, 16, 0, 0),
        # compaction of a fragmented pool: pages move down, all tables follow
        _pages("compact-1200", 6, 2600, 1200, 8, 128, 32, 130, 21),
        # one decode step's answer: eight rows with twenty alternatives, an odd vocabulary
        _logprobs("answer-8x50257", 8, 50257, "fp32", 20),
        # scoring a text (perplexity): every position's token
        _logprobs("score-3000x131072", 3000, 131072, "bf16", 5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "pages", "logprobs"])
    if op in ("attention", "append"):
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
        head_dim = rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128])
        seqs = _log_int(rng, 1, 96)
        # tokens and positions in all stay below the largest listed case's
        new_hi = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, max(18, 4000 // seqs))])
        len_hi = _log_int(rng, max(40, new_hi), max(60, new_hi, min(100000 if new_hi <= 16 else 12000, 250000 // seqs)))
        len_lo = max(1, _log_int(rng, 1, len_hi))
        new_lo = _log_int(rng, 1, new_hi)
        if op == "append":
            return {k: v for k, v in _append("", seqs, (new_lo, new_hi), (len_lo, len_hi), heads, kv_heads, head_dim,
                                             page, rng.randrange(1 << 30)).items() if k != "name"}
        masked = rng.random() < 0.4
        c = _attention("", seqs, (new_lo, new_hi), (len_lo, len_hi), heads, kv_heads, head_dim, page,
                       rng.randrange(1 << 30),
                       softcap=rng.choice([0.0, 20.0, 50.0]) if masked else 0.0,
                       slopes=masked and rng.random() < 0.5,
                       window=_log_int(rng, 16, 4000) if masked and rng.random() < 0.5 else 0,
                       prefix=_log_int(rng, 1, 300) if masked and rng.random() < 0.5 else 0)
    elif op == "pages":
        layers = _log_int(rng, 1, 40)
        page, kv_heads, head_dim = rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        per = layers * page * kv_heads * head_dim * 4
        pages = _log_int(rng, 8, max(16, min(4000, (3 << 29) // per)))
        moves = _log_int(rng, 1, pages // 2)
        rows = rng.choice([0, _log_int(rng, 1, 200)])
        c = _pages("", layers, pages, moves, kv_heads, head_dim, page, rows, _log_int(rng, 1, 300) if rows else 0)
    else:
        vocab = _log_int(rng, 1000, 160000)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        rows = _log_int(rng, 1, max(2, min(4000, (700 << 20) // (vocab * 4))))
        c = _logprobs("", rows, vocab, dtype, rng.choice([0, 1, 5, 20, 32]))
    return {k: v for k, v in c.items() if k != "name"}


def _lens(case):
    """New tokens and positions of every sequence: a new token count never above the length."""
    r = random.Random(case["lens_seed"])
    new, length = [], []
    for _ in range(case["seqs"]):
        n = _log_int(r, case["new_lo"], case["new_hi"])
        length.append(max(n, _log_int(r, case["len_lo"], case["len_hi"])))
        new.append(n)
    return new, length


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _page_table(length, page, seed):
    """Pages of every sequence, scattered over a pool with a few unused pages; -1 past the end."""
    r = random.Random(seed)
    need = [-(-n // page) for n in length]
    pool = sum(need) + 5
    order = list(range(pool))
    r.shuffle(order)
    table = torch.full((len(length), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at: at + n], dtype=torch.int32)
        at += n
    return table.cuda(), pool


def _starts(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def _slopes(heads):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op in ("attention", "append"):
        new, length = _lens(case)
        H, Hkv, D, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
        N = sum(new)
        st["new"], st["length"], st["starts"] = new, length, _starts(new)
        st["table"], pool = _page_table(length, page, seed)
        st["q_start"] = torch.tensor(st["starts"], dtype=torch.int32).cuda()
        st["kv_len"] = torch.tensor(length, dtype=torch.int32).cuda()
        # normalised keys (unit RMS, as a per-head norm leaves them) and values of mixed size
        st["k"] = torch.randn(pool, page, Hkv, D, generator=g, device="cuda", dtype=BF16)
        st["v"] = torch.randn(pool, page, Hkv, D, generator=g, device="cuda", dtype=BF16)
    if op == "attention":
        st["q"] = (1.5 * torch.randn(N, H * D, generator=g, device="cuda")).to(BF16)
        st["slopes"] = _slopes(H).cuda() if case["slopes"] else None
        st["prefix"] = None
        st["prefix_len"] = [0] * len(new)
        if case["prefix"]:
            r = random.Random(seed + 1)
            st["prefix_len"] = [r.randint(0, case["prefix"]) for _ in new]
            st["prefix"] = torch.tensor(st["prefix_len"], dtype=torch.int32).cuda()
        if own:
            import online_activation_aware_b200 as ttq

            st["plan"] = ttq.AttentionPlan(len(new), N, H, Hkv, D, max_new=max(new))
    elif op == "append":
        # a stacked projection's output and the norm weights; the rotary table of the positions
        st["qkv"] = torch.randn(N, (H + 2 * Hkv) * D, generator=g, device="cuda").to(BF16)
        st["wq"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF16)
        st["wk"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF16)
        ang = torch.arange(max(length), dtype=torch.float64)[:, None] * 1.0e6 ** (
            -torch.arange(0, D, 2, dtype=torch.float64) / D)[None]
        st["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float().cuda()
    elif op == "pages":
        shape = (case["layers"], case["pages"], case["page"], case["kv_heads"], case["head_dim"])
        st["k"] = torch.randn(shape, generator=g, device="cuda", dtype=BF16)
        st["v"] = torch.randn(shape, generator=g, device="cuda", dtype=BF16)
        r = random.Random(seed)
        pick = r.sample(range(case["pages"]), 2 * case["moves"])
        src, dst = pick[: case["moves"]], pick[case["moves"]:]
        if case["rows"] == 0:  # branches of one prompt: every copy reads the same page
            src = [src[0]] * len(src)
        st["src"] = torch.tensor(src, dtype=torch.int32).cuda()
        st["dst"] = torch.tensor(dst, dtype=torch.int32).cuda()
        if case["rows"]:
            mapping = torch.arange(case["pages"], dtype=torch.int32)
            mapping[torch.tensor(src)] = torch.tensor(dst, dtype=torch.int32)
            st["mapping"] = mapping.cuda()
            table = torch.randint(0, case["pages"], (case["rows"], case["width"]), generator=g, device="cuda")
            ends = torch.randint(1, case["width"] + 1, (case["rows"], 1), generator=g, device="cuda")
            cols = torch.arange(case["width"], device="cuda")[None]
            st["table"] = torch.where(cols < ends, table, -1).to(torch.int32)
    else:
        V = case["vocab"]
        # logits of a language model: a broad bulk and a few raised tokens a row
        x = 2.0 * torch.randn(case["rows"], V, generator=g, device="cuda")
        hot = torch.randint(0, V, (case["rows"], 12), generator=g, device="cuda")
        x.scatter_add_(1, hot, 12.0 * torch.rand(case["rows"], 12, generator=g, device="cuda"))
        st["logits"] = x.to(DTYPES[case["dtype"]])
        # scored tokens: mostly likely ones, some rows without a token (padding)
        tok = torch.where(torch.rand(case["rows"], generator=g, device="cuda") < 0.7, hot[:, 0],
                          torch.randint(0, V, (case["rows"],), generator=g, device="cuda"))
        st["tokens"] = torch.where(torch.rand(case["rows"], generator=g, device="cuda") < 0.05, -1, tok)
    return st


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "append": _own_append, "pages": _own_pages,
                "logprobs": _own_logprobs}[op](state)
    return {"attention": _plain_attention, "append": _plain_append, "pages": _plain_pages,
            "logprobs": _plain_logprobs}[op](state)


def _own_attention(st):
    import online_activation_aware_b200 as ttq

    c = st["case"]
    st["plan"].update(st["q_start"], st["kv_len"], window=c["window"], prefix=st["prefix"])
    return ttq.paged_attention(st["q"], st["plan"], st["k"], st["v"], st["table"], softcap=c["softcap"],
                               slopes=st["slopes"])


def _own_append(st):
    import online_activation_aware_b200 as ttq

    c = st["case"]
    q = ttq.qk_norm_rope_paged(st["qkv"], c["heads"], c["kv_heads"], c["head_dim"], st["wq"], st["wk"], 1e-6, st["rope"],
                               st["q_start"], st["kv_len"], st["k"], st["v"], st["table"])
    return {"q": q, "k": st["k"], "v": st["v"]}


def _own_pages(st):
    import online_activation_aware_b200 as ttq

    ttq.copy_pages(st["k"], st["v"], st["src"], st["dst"])
    out = {"k": st["k"], "v": st["v"]}
    if st["case"]["rows"]:
        out["table"] = ttq.remap_pages(st["table"], st["mapping"])
    return out


def _own_logprobs(st):
    import online_activation_aware_b200 as ttq

    return ttq.token_logprobs(st["logits"], st["tokens"], top=st["case"]["top"])


def _plain_attention(st):
    c = st["case"]
    H, Hkv, D = c["heads"], c["kv_heads"], c["head_dim"]
    G = H // Hkv
    outs = []
    for b, (n, L) in enumerate(zip(st["new"], st["length"])):
        pages = st["table"][b, : -(-L // c["page"])].long()
        k = st["k"][pages].reshape(-1, Hkv, D)[:L].float()
        v = st["v"][pages].reshape(-1, Hkv, D)[:L].float()
        q = st["q"][st["starts"][b]: st["starts"][b + 1]].float().view(n, Hkv, G, D)
        kpos = torch.arange(L, device="cuda")
        step = max(1, (1 << 28) // (L * H))  # rows at a time: bounded scores
        rows = []
        for i in range(0, n, step):
            qi = q[i: i + step]
            qpos = L - n + i + torch.arange(qi.shape[0], device="cuda")
            s = torch.einsum("nhgd,khd->hgnk", qi, k) / math.sqrt(D)
            if c["softcap"]:
                s = c["softcap"] * torch.tanh(s / c["softcap"])
            if st["slopes"] is not None:
                s = s + st["slopes"].view(Hkv, G, 1, 1) * (kpos[None] - qpos[:, None]).float()
            seen = kpos[None] <= qpos[:, None]
            if c["window"]:
                seen = seen & (kpos[None] > qpos[:, None] - c["window"])
            seen = seen | (kpos[None] < st["prefix_len"][b])
            s = s.masked_fill(~seen, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.einsum("hgnk,khd->nhgd", p, v) / p.sum(-1).permute(2, 0, 1).unsqueeze(-1)
            rows.append(o.reshape(-1, H * D))
        outs.append(torch.cat(rows).to(BF16))
    return torch.cat(outs)


def _positions(st):
    """Sequence and position of every new token."""
    seq = torch.tensor([b for b, n in enumerate(st["new"]) for _ in range(n)], device="cuda")
    pos = torch.tensor([L - n + i for n, L in zip(st["new"], st["length"]) for i in range(n)], device="cuda")
    return seq, pos


def _norm_rope(x, w, eps, cos, sin):
    y = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w
    a, b = y.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(st):
    c = st["case"]
    H, Hkv, D = c["heads"], c["kv_heads"], c["head_dim"]
    seq, pos = _positions(st)
    x = st["qkv"].float().view(-1, H + 2 * Hkv, D)
    cos, sin = st["rope"][pos, None, :, 0], st["rope"][pos, None, :, 1]
    q = _norm_rope(x[:, :H], st["wq"].float(), 1e-6, cos, sin).to(BF16)
    k = _norm_rope(x[:, H: H + Hkv], st["wk"].float(), 1e-6, cos, sin).to(BF16)
    page = st["table"][seq, pos // c["page"]].long()
    st["k"][page, pos % c["page"]] = k
    st["v"][page, pos % c["page"]] = st["qkv"].view(-1, H + 2 * Hkv, D)[:, H + Hkv:]
    return {"q": q.reshape(-1, H * D), "k": st["k"], "v": st["v"]}


def _plain_pages(st):
    src, dst = st["src"].long(), st["dst"].long()
    for t in (st["k"], st["v"]):
        t[:, dst] = t[:, src]
    out = {"k": st["k"], "v": st["v"]}
    if st["case"]["rows"]:
        t = st["table"]
        out["table"] = torch.where(t >= 0, st["mapping"][t.clamp(min=0).long()], t)
    return out


def _ordered(x):
    """int64 keys in the order of the values, ties to the lowest index; keys are distinct."""
    b = x.contiguous().view(torch.int32)
    b = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
    V = x.shape[-1]
    return (b << 20) | (V - 1 - torch.arange(V, device=x.device))


def _plain_logprobs(st):
    top, tokens = st["case"]["top"], st["tokens"]
    outs = []
    N, V = st["logits"].shape
    step = max(1, (1 << 27) // V)
    for i in range(0, N, step):
        x = st["logits"][i: i + step].float()
        t = tokens[i: i + step]
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        s = e.sum(-1, keepdim=True)
        lse = m + torch.log(s)
        lp = torch.where(t >= 0, x.gather(1, t.clamp(min=0)[:, None])[:, 0] - lse[:, 0], 0.0)
        ent = torch.log(s)[:, 0] - (e * (x - m)).sum(-1) / s[:, 0]
        one = [lp, ent]
        if top:
            key = torch.topk(_ordered(x), top, dim=-1).values
            ids = V - 1 - (key & ((1 << 20) - 1))
            one += [ids, x.gather(1, ids) - lse]
        outs.append(one)
    names = ["logprob", "entropy"] + (["top_ids", "top_logprobs"] if top else [])
    return {n: torch.cat([o[j] for o in outs]) for j, n in enumerate(names)}


# ------------------------------------------------------------------ what a pass cannot do without


def _visible(case, n, L):
    """Visible (token, position) pairs of a sequence, its prefix apart (a few positions)."""
    w = case["window"]
    p0 = L - n
    if not w:
        return n * p0 + n * (n + 1) // 2
    return sum(min(p0 + i + 1, w) for i in range(n))


def work(case):
    op = case["op"]
    if op in ("attention", "append"):
        new, length = _lens(case)
        H, Hkv, D = case["heads"], case["kv_heads"], case["head_dim"]
        N = sum(new)
        if op == "append":
            row = (H + 2 * Hkv) * D
            return {"bytes": N * row * 2 * 2 + 4 * N * D, "flops": N * (H + Hkv) * D * 8}
        pairs = sum(_visible(case, n, L) for n, L in zip(new, length))
        read = sum(min(L, n + case["window"] - 1) if case["window"] else L for n, L in zip(new, length))
        return {"bytes": read * Hkv * D * 2 * 2 + N * H * D * 2 * 2 + 4 * -(-read // case["page"]),
                "flops": pairs * H * D * 4}
    if op == "pages":
        page = case["layers"] * case["page"] * case["kv_heads"] * case["head_dim"] * 2 * 2
        read = 1 if case["rows"] == 0 else case["moves"]  # a fork reads one page for all branches
        return {"bytes": page * (read + case["moves"]) + 8 * case["moves"] + 8 * case["rows"] * case["width"], "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    n = case["rows"] * case["vocab"]
    return {"bytes": n * size + case["rows"] * (16 + 12 * case["top"]), "flops": 6 * n}


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "pages": _exact_pages,
            "logprobs": _exact_logprobs}[case["op"]](st)


def _exact_attention(st):
    c = st["case"]
    H, Hkv, D, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    N = st["q"].shape[0]
    out = torch.zeros(N, H, D, dtype=torch.float64, device="cuda")
    q = st["q"].view(N, H, D)
    for b in range(c["seqs"]):
        a, n, L = st["starts"][b], st["new"][b], st["length"][b]
        j = torch.arange(L, device="cuda")
        where = st["table"][b].long()[j // page]
        for kh in range(Hkv):
            K = st["k"][where, j % page, kh].double()
            V = st["v"][where, j % page, kh].double()
            for h in range(kh * (H // Hkv), (kh + 1) * (H // Hkv)):
                for i in range(0, n, 2048):
                    m = min(n, i + 2048)
                    pos = torch.arange(L - n + i, L - n + m, device="cuda")[:, None]
                    z = q[a + i: a + m, h].double() @ K.T * D ** -0.5
                    if c["softcap"] > 0:
                        z = torch.tanh(z / c["softcap"]) * c["softcap"]
                    if c["slopes"]:
                        z = z - 2.0 ** (-8.0 * (h + 1) / H) * (pos - j)
                    hidden = (j > pos) | ((j <= pos - c["window"]) if c["window"] else torch.zeros_like(j > pos))
                    hidden &= j >= st["prefix_len"][b]
                    z[hidden] = -math.inf
                    out[a + i: a + m, h] = torch.softmax(z, -1) @ V
    return out.view(N, H * D)


def _exact_append(st):
    c = st["case"]
    H, Hkv, D, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    N = st["qkv"].shape[0]
    x = st["qkv"].double().view(N, H + 2 * Hkv, D)
    q = torch.empty(N, H, D, dtype=torch.float64, device="cuda")
    k, v = st["k"].double(), st["v"].double()
    for b in range(c["seqs"]):
        a, n, L = st["starts"][b], st["new"][b], st["length"][b]
        p = torch.arange(L - n, L, device="cuda")
        turn = torch.complex(st["rope"][p, :, 0].double(), st["rope"][p, :, 1].double())[:, None]
        y = x[a: a + n]

        def spin(part, w):
            r = part / (part.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
            z = torch.complex(r[..., : D // 2].contiguous(), r[..., D // 2:].contiguous()) * turn
            return torch.cat([z.real, z.imag], -1)

        q[a: a + n] = spin(y[:, :H], st["wq"])
        at = st["table"][b].long()[p // page]
        k[at, p % page] = spin(y[:, H: H + Hkv], st["wk"])
        v[at, p % page] = y[:, H + Hkv:]
    return {"q": q.view(N, H * D), "k": k, "v": v}


def _exact_pages(st):
    out = {}
    for name in ("k", "v"):
        t = st[name]
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            t[:, d].copy_(t[:, s])
        out[name] = t
    if st["case"]["rows"]:
        to = dict(enumerate(st["mapping"].tolist()))
        out["table"] = torch.tensor([[to.get(p, -1) for p in row] for row in st["table"].tolist()], dtype=torch.int32,
                                    device="cuda")
    return out


def _exact_logprobs(st):
    top, rows = st["case"]["top"], st["logits"].shape[0]
    res = {"logprob": [], "entropy": [], "top_ids": [], "top_logprobs": []}
    step = max(1, (1 << 25) // st["logits"].shape[1])
    for i in range(0, rows, step):
        x = st["logits"][i: i + step].double()
        lp = x - torch.logsumexp(x, -1, keepdim=True)
        t = st["tokens"][i: i + step]
        got = lp[torch.arange(len(t), device="cuda"), t.clamp(min=0)]
        res["logprob"].append(torch.where(t < 0, torch.zeros_like(got), got))
        res["entropy"].append(-(lp.exp() * lp).sum(-1))
        if top:
            order = torch.sort(lp, dim=-1, descending=True, stable=True)
            res["top_ids"].append(order.indices[:, :top].clone())
            res["top_logprobs"].append(order.values[:, :top].clone())
    return {k: torch.cat(v) for k, v in res.items() if v}
