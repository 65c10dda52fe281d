"""Float64 oracle of attention with a sliding window and sinks and of its paged cache (test
infrastructure only; shares nothing with the HIP path).

The query at position p of its sequence sees the keys j <= p with j > p - window or j < sinks."""
from __future__ import annotations

import numpy as np


def _bounds(n, L, cu):
    if cu is None:
        return [(b, 0, L) for b in range(n)]
    return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def visible(nq, nk, window, sinks):
    """(nq, nk): the queries are the last positions of nk keys."""
    p = np.arange(nq)[:, None] + (nk - nq)
    j = np.arange(nk)[None, :]
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def _probs(Q, K, see, scale):
    s = np.where(see, scale * (Q @ K.T), -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    e = np.where(see, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    z = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(z > 0, np.log(z) + np.where(np.isfinite(top), top, 0.0), -np.inf)
    return e / np.where(z > 0, z, 1.0), lse[:, 0]


def attention(q, k, v, *, window=0, sinks=0, scale=None, cu=None, cu_k=None):
    """o (n, L, H, D) and lse (n, L, H); rows of no sequence are NaN."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, L, H, D = q.shape
    g = H // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    for (b, q0, q1), (_, k0, k1) in zip(_bounds(n, L, cu), _bounds(n, k.shape[1], cu if cu_k is None else cu_k)):
        see = visible(q1 - q0, k1 - k0, window, sinks)
        for h in range(H):
            P, z = _probs(q[b, q0:q1, h], k[b, k0:k1, h // g], see, scale)
            o[b, q0:q1, h] = P @ v[b, k0:k1, h // g]
            lse[b, q0:q1, h] = z
    return o, lse


def attention_backward(q, k, v, do, *, o=None, window=0, sinks=0, scale=None, cu=None, cu_k=None):
    """dict of the gradients q, k, v; rows of no sequence are zero.  o: the forward's result as it was stored (its
    own by default): dS = P (do.v - do.o), and 0 for a query that sees one key."""
    q, k, v, do = (np.asarray(t, np.float64) for t in (q, k, v, do))
    n, L, H, D = q.shape
    g = H // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    o = attention(q, k, v, window=window, sinks=sinks, scale=scale, cu=cu, cu_k=cu_k)[0] if o is None else np.asarray(o, np.float64)
    out = {"q": np.zeros_like(q), "k": np.zeros_like(k), "v": np.zeros_like(v)}
    for (b, q0, q1), (_, k0, k1) in zip(_bounds(n, L, cu), _bounds(n, k.shape[1], cu if cu_k is None else cu_k)):
        see = visible(q1 - q0, k1 - k0, window, sinks)
        lone = see.sum(-1, keepdims=True) == 1
        for h in range(H):
            u = h // g
            Q, K, V, dO = q[b, q0:q1, h], k[b, k0:k1, u], v[b, k0:k1, u], do[b, q0:q1, h]
            P, _ = _probs(Q, K, see, scale)
            dS = np.where(lone, 0.0, P * (dO @ V.T - (dO * o[b, q0:q1, h]).sum(-1, keepdims=True)))
            out["q"][b, q0:q1, h] = scale * (dS @ K)
            out["k"][b, k0:k1, u] += scale * (dS.T @ Q)
            out["v"][b, k0:k1, u] += P.T @ dO
    return out


# ---------------------------------------------------------------- the cache

def e4m3(x):
    """Values of 8 bits (3 of fraction, least exponent 2^-6) nearest to x, ties to even; |x| <= 448.
    Infinities and NaN become NaN."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    y = np.where(fin, x, 0.0)
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.where(fin, np.round(y / step) * step, np.nan)


def page_scale(x):
    """The least power of two s with |x| <= 448 s for every finite value; 2^-100 at least."""
    x = np.abs(np.asarray(x, np.float64))
    top = np.where(np.isfinite(x), x, 0.0).max(initial=0.0)
    if top == 0.0:
        return 2.0 ** -100
    m, e = np.frexp(top / 448.0)  # top / 448 = m 2^e, m in [0.5, 1)
    return max(2.0 ** -100, 2.0 ** (e - 1 if m == 0.5 else e))


def cache_write(k, cache, scale, table, lens, cu=None):
    """One of the two caches (pages, Hk, page, D) as values of its codes, with its scales or None: the new tokens
    (n, L, Hk, D) behind the lens that the sequences hold.  Returns both."""
    k = np.asarray(k, np.float64)
    cache = np.array(cache, np.float64)
    scale = None if scale is None else np.array(scale, np.float64)
    pages, hk, page, _ = cache.shape
    for i, (b, t0, t1) in enumerate(_bounds(k.shape[0], k.shape[1], cu)):
        held, n = int(lens[i]), t1 - t0
        for e in range(held // page, -(-(held + n) // page) if n else 0):
            if e >= table.shape[1] or not 0 <= table[i, e] < pages:
                continue
            lo, hi = max(held, e * page), min(held + n, (e + 1) * page)
            a, z = lo - e * page, hi - e * page
            for h in range(hk):
                new, rows = k[b, t0 + lo - held:t0 + hi - held, h], cache[table[i, e], h]
                if scale is None:
                    rows[a:z] = new
                    continue
                s = page_scale(new)
                if a > 0:
                    had = scale[table[i, e], h]
                    s = max(s, had)
                    rows[:a] = e4m3(rows[:a] * (had / s))
                rows[a:z] = e4m3(new / s)
                scale[table[i, e], h] = s
    return cache, scale


def decode_step(q, k_cache, v_cache, table, lens, *, k_scale=None, v_scale=None, window=0, sinks=0, scale=None):
    """o (n, H, D): the query of each sequence over the values in its pages; keys of pages out of range are left out."""
    q = np.asarray(q, np.float64)
    n, H, D = q.shape
    pages, hk, page, _ = k_cache.shape
    g = H // hk
    scale = D ** -0.5 if scale is None else scale
    o = np.zeros(q.shape)
    for i in range(n):
        held = min(max(int(lens[i]), 0), table.shape[1] * page)
        j = np.arange(held)
        if window:
            j = j[(j >= held - window) | (j < sinks)]
        at = table[i, j // page]
        j = j[(at >= 0) & (at < pages)]
        at, row = table[i, j // page], j % page
        for h in range(H):
            K, V = (np.asarray(c, np.float64)[at, h // g, row] for c in (k_cache, v_cache))
            if k_scale is not None:
                K, V = K * np.asarray(k_scale, np.float64)[at, h // g][:, None], V * np.asarray(v_scale, np.float64)[at, h // g][:, None]
            P, _ = _probs(q[i, h][None], K, np.ones((1, len(j)), bool), scale)
            o[i, h] = (P @ V)[0]
    return o
