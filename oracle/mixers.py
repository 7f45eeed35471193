"""Float64 restatement of the mixers between the packed linears, from their formulas: the paged
K/V cache's plan and writes, attention over the cache and over packed prompts, and the gated delta
rule as the token-by-token recurrence.  NumPy only; shares nothing with the library.

Each attention and delta function also returns the magnitudes from which the tests derive their
tolerances (sums of absolute terms of the same formulas).
"""
from __future__ import annotations

import numpy as np


def cache_plan(cached, fresh, page, free, table, T):
    """(table, slots [T], row_start, total, used): a step's new pages, in order, from ``free``."""
    table = np.array(table, dtype=np.int32)
    B, width = table.shape
    slots = np.full(T, -1, dtype=np.int64)
    row_start = np.zeros(B + 1, dtype=np.int64)
    taken = t = 0
    for b in range(B):
        c, f = int(cached[b]), int(fresh[b])
        have, need = -(-c // page), -(-(c + f) // page)
        for p in range(min(have, width), min(need, width)):
            table[b, p] = free[taken] if taken < len(free) else -1
            taken += 1
        for pos in range(c, c + f):
            if t < T and pos // page < width and table[b, pos // page] >= 0:
                slots[t] = int(table[b, pos // page]) * page + pos % page
            t += 1
        row_start[b + 1] = t
    return table, slots, row_start.astype(np.int32), (np.asarray(cached) + np.asarray(fresh)).astype(np.int32), min(taken, len(free))


def cache_write(k, v, slots, k_cache, v_cache):
    """Copies of the caches [pages, H, page, D] with every token of a slot >= 0 written."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    page = k_cache.shape[2]
    for t, s in enumerate(slots):
        if 0 <= s < k_cache.shape[0] * page:
            k_cache[s // page, :, s % page] = k[t]
            v_cache[s // page, :, s % page] = v[t]
    return k_cache, v_cache


def _attend(q, k, v, seen, scale):
    """One head of one request: q [n, D], k, v [L, D], seen [n, L] -> o [n, D] and the tolerance's
    parts: sum w |v|, sum |v| / (sum of weights over the largest), and max |score terms|."""
    n, D = q.shape
    o = np.zeros((n, D))
    wv = np.zeros((n, D))
    tail = np.zeros((n, D))
    sterm = np.zeros((n, 1))
    for i in range(n):
        at = np.flatnonzero(seen[i])
        if not len(at):
            continue
        s = (k[at] @ q[i]) * scale
        w = np.exp(s - s.max())
        o[i] = w @ v[at] / w.sum()
        wv[i] = w @ np.abs(v[at]) / w.sum()
        tail[i] = np.abs(v[at]).sum(0) / w.sum()
        sterm[i] = (np.abs(k[at]) @ np.abs(q[i])).max() * scale
    return o, wv, tail, sterm


def attention_tolerance(o, wv, tail, sterm, D):
    """Half an fp16 ulp of the output; weights that were rounded to fp16 for the product with v
    (2^-11 of each, 2^-25 where it is below fp16's normal range) and their sum in fp32 (another
    2^-11 covers it); scores as fp32 sums of D products (D 2^-24 of the absolute terms, twice: in a
    weight and in the sum)."""
    return 2.0 ** -11 * np.abs(o) + (2.0 ** -10 + 2 * D * 2.0 ** -24 * sterm) * wv + 2.0 ** -25 * (tail + 1)


def prompt_attention(q, k, v, q_start, k_start, scale):
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    Hq, D = q.shape[1:]
    G = Hq // k.shape[1]
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(q_start) - 1):
        q0, q1, k0, k1 = q_start[b], q_start[b + 1], k_start[b], k_start[b + 1]
        seen = np.arange(k1 - k0)[None, :] <= np.arange(q1 - q0)[:, None] + (k1 - k0) - (q1 - q0)
        for h in range(Hq):
            r = _attend(q[q0:q1, h], k[k0:k1, h // G], v[k0:k1, h // G], seen, scale)
            o[q0:q1, h] = r[0]
            tol[q0:q1, h] = attention_tolerance(*r, D)
    return o, tol


def tree_attention(q, k_cache, v_cache, table, total, row_start, tree, scale):
    q = np.asarray(q, dtype=np.float64)
    Hq, D = q.shape[1:]
    pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(total)):
        r0, r1, L = int(row_start[b]), int(row_start[b + 1]), int(total[b])
        n = r1 - r0
        if n == 0:
            continue
        pos = np.arange(L)
        pg = np.asarray(table)[b, pos // page]
        ok = (pg >= 0) & (pg < pages)
        seen = np.zeros((n, L), dtype=bool)
        for i in range(n):
            word = (1 << (i + 1)) - 1 if tree is None else int(tree[r0 + i]) & (2 ** 64 - 1)
            seen[i, : L - n] = True
            seen[i, L - n:] = [bool(word >> j & 1) for j in range(n)]
        seen &= ok[None, :]
        at = np.where(ok, pg, 0)
        for h in range(Hq):
            k = k_cache[at, h // G, pos % page].astype(np.float64)
            v = v_cache[at, h // G, pos % page].astype(np.float64)
            r = _attend(q[r0:r1, h], k, v, seen, scale)
            o[r0:r1, h] = r[0]
            tol[r0:r1, h] = attention_tolerance(*r, D)
    return o, tol


def gated_delta(q, k, v, g, beta, row_start, state, normalise, scale):
    """The recurrence; state [B, Hv, D, D].  Returns (o, final states, sum of |terms| of o): the
    last is scale |q| . M with M the state's terms added up without signs."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    g, beta = np.asarray(g, dtype=np.float64), np.asarray(beta, dtype=np.float64)
    T, Hk, D = q.shape
    Hv = v.shape[1]
    if normalise:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) for x in (q, k))
    q, k = np.repeat(q, Hv // Hk, 1), np.repeat(k, Hv // Hk, 1)
    state = np.array(state, dtype=np.float64)
    o, mag = np.zeros((T, Hv, D)), np.zeros((T, Hv, D))
    for b in range(len(row_start) - 1):
        S = state[b]
        M = np.abs(S)
        for t in range(row_start[b], row_start[b + 1]):
            a = np.exp(g[t])[:, None, None]
            S = a * S
            u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            M = a * M + np.abs(k[t][:, :, None] * u[:, None, :])
            o[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
            mag[t] = scale * np.einsum("hkv,hk->hv", M, np.abs(q[t]))
        state[b] = S
    return o, state, mag
