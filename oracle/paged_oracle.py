"""Plain fp64 oracle (numpy) of the paged-cache operators: attention of several sequences' new
tokens over pages, the page writes of new keys and values, page copies and table rewrites,
and token log probabilities. Test infrastructure only."""

import numpy as np

from oracle import decoder_oracle as DO


def gather(pool, row, length):
    """Positions 0 .. length-1 of a sequence: pool [pages, page_size, heads, D], row its table."""
    ps = pool.shape[1]
    p = np.arange(length)
    return pool[row[p // ps], p % ps]


def visible(n, L, window=0, prefix=0):
    """[n, L] truth: position k is visible to new token i (at position L - n + i)."""
    pos = (L - n + np.arange(n))[:, None]
    k = np.arange(L)[None]
    seen = k <= pos
    if window:
        seen &= k > pos - window
    return seen | (k < prefix)


def attention(q, k_pages, v_pages, table, new, length, softcap=0.0, slopes=None, window=0, prefix=None):
    """q [tokens, H, D]. Returns (out [sum new, H, D], weighted |v| of the same shape: the sum
    of softmax weights times |v|, the scale on which rounding of the weights acts)."""
    H, D = q.shape[1:]
    Hkv = k_pages.shape[2]
    outs, mags = [], []
    at = 0
    for b, (n, L) in enumerate(zip(new, length)):
        qb = q[at: at + n]
        at += n
        o, a = np.zeros((n, H, D)), np.zeros((n, H, D))
        if L > 0 and n > 0:
            pre = 0 if prefix is None else min(prefix[b], L)
            seen = visible(n, L, window, pre)
            need = seen.any(0)                     # positions no token sees may hold anything
            pos = (L - n + np.arange(n))[:, None]
            ps = k_pages.shape[1]
            K = np.zeros((L, Hkv, D))
            V = np.zeros((L, Hkv, D))
            kk = np.arange(L)[need]
            K[need] = k_pages[table[b][kk // ps], kk % ps]
            V[need] = v_pages[table[b][kk // ps], kk % ps]
            for h in range(H):
                kh = h // (H // Hkv)
                s = qb[:, h] @ K[:, kh].T / np.sqrt(D)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s + slopes[h] * (np.arange(L)[None] - pos)
                s = np.where(seen, s, -np.inf)
                m = s.max(1, keepdims=True)
                w = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
                l = w.sum(1, keepdims=True)
                w = np.divide(w, l, out=np.zeros_like(w), where=l > 0)
                o[:, h] = w @ V[:, kh]
                a[:, h] = w @ np.abs(V[:, kh])
        outs.append(o)
        mags.append(a)
    return np.concatenate(outs), np.concatenate(mags)


def append(qkv, H, Hkv, D, wq, wk, new, length, table, page_size, base=1.0e6, eps=1e-6):
    """Returns q [sum new, H, D], and lists of (page, slot, k [Hkv, D], v [Hkv, D])."""
    x = qkv.reshape(qkv.shape[0], H + 2 * Hkv, D)
    q, writes = [], []
    t = 0
    for b, (n, L) in enumerate(zip(new, length)):
        for i in range(n):
            pos = np.array([L - n + i])
            q.append(DO.rope(DO.rmsnorm(x[t: t + 1, :H], wq, eps), pos, base)[0])
            k = DO.rope(DO.rmsnorm(x[t: t + 1, H: H + Hkv], wk, eps), pos, base)[0]
            writes.append((int(table[b][pos[0] // page_size]), int(pos[0] % page_size), k, x[t, H + Hkv:]))
            t += 1
    return np.array(q).reshape(-1, H, D), writes


def logprobs(x, tokens, top):
    """x fp64 [rows, vocab]. Rows with NaN, +inf or nothing but -inf have NaN probabilities."""
    rows, V = x.shape
    m = x.max(1)
    ok = np.isfinite(m) & ~np.isnan(x).any(1)
    mm = np.where(ok, m, 0.0)[:, None]
    with np.errstate(all="ignore"):
        e = np.exp(np.where(ok[:, None], x - mm, -np.inf))
        s = e.sum(1)
        lse = np.where(ok, mm[:, 0] + np.log(s), np.nan)
        lp = x - lse[:, None]
        ent = np.where(ok, -(np.where(e > 0, lp, 0.0) * e).sum(1) / s, np.nan)
    got = np.array([0.0 if t < 0 else lp[r, t] for r, t in enumerate(tokens)])
    key = np.where(np.isnan(x), -np.inf, x)
    order = np.zeros((rows, top), dtype=np.int64)
    for r in range(rows):
        # falling value, NaN after -inf, ties by rising index
        order[r] = np.lexsort((np.arange(V), np.isnan(x[r]), -key[r]))[:top]
    return got, ent, order, np.take_along_axis(lp, order, 1)
