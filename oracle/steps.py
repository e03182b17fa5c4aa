"""Plain fp64 restatements of the operators around a beam step (numpy, one row or head at a time): logits
processing, the choice of the beams, their bookkeeping, the keys' attention weights and the eviction of cached
rows. They share no code with the library."""
from __future__ import annotations

import numpy as np


def process_row(x, prompt=(), tokens=(), repetition=None, frequency=None, presence=None, bias=(), temperature=None,
                allowed=None):
    """One row of logits (fp64 in, fp64 out). bias: (token, value) pairs in list order; allowed: bool [vocab]."""
    x = np.array(x, np.float64)
    V = len(x)
    made = [int(t) for t in tokens if 0 <= t < V]
    if repetition is not None:
        for t in set(made) | {int(t) for t in prompt if 0 <= t < V}:
            x[t] = x[t] / repetition if x[t] > 0 else x[t] * repetition
    for t in set(made):
        if frequency is not None:
            x[t] -= frequency * made.count(t)
        if presence is not None:
            x[t] -= presence
    seen = set()
    for t, v in bias:
        if 0 <= t < V and t not in seen:
            seen.add(t)
            x[t] += v
    if temperature is not None:
        x = x / temperature
    if allowed is not None:
        x[~np.asarray(allowed, bool)] = -np.inf
    return x


def log_sum_exp(x):
    x = np.asarray(x, np.float64)
    m = x.max() if len(x) else -np.inf
    if np.isnan(x).any():
        return np.nan
    if np.isinf(m):
        return m
    return m + np.log(np.exp(x - m).sum())


def unpack_mask(words, vocab):
    w = np.asarray(words).view(np.uint32)
    return ((w[:, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(-1)[:vocab].astype(bool)


def pack_mask(allowed):
    """bool [states, vocab] -> int32 [states, ceil(vocab / 32)]"""
    a = np.asarray(allowed, bool)
    n = -(-a.shape[1] // 32)
    full = np.zeros((a.shape[0], n * 32), np.uint64)
    full[:, :a.shape[1]] = a
    return (full.reshape(a.shape[0], n, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def select(x, lse, cum, num, allowed=None):
    """One request: x fp32 [W, V], lse and cum fp32 [W]; allowed bool [W, V] or None. The scores are the two fp32
    operations of the definition; the order is exact."""
    x, lse, cum = (np.asarray(a, np.float32) for a in (x, lse, cum))
    W, V = x.shape
    with np.errstate(invalid="ignore"):
        s = ((x - lse[:, None]) + cum[:, None]).astype(np.float32)
    ok = s > -np.inf
    if allowed is not None:
        ok &= allowed
    flat = np.flatnonzero(ok.reshape(-1))
    v = s.reshape(-1)[flat]
    order = np.lexsort((flat, -(v.astype(np.float64))))[:num]
    scores = np.full(num, -np.inf, np.float32)
    parents = np.full(num, -1, np.int32)
    tokens = np.full(num, -1, np.int32)
    scores[:len(order)] = v[order]
    parents[:len(order)] = flat[order] // V
    tokens[:len(order)] = flat[order] % V
    return scores, parents, tokens


def advance(parents, chosen, P, T, ci, tokens):
    """One request: ci [W, max_seq] and tokens [W, n] re-ordered; returns the new tables."""
    W = len(parents)
    ci2, tok2 = ci.copy(), tokens.copy()
    for w in range(W):
        p = parents[w] if 0 <= parents[w] < W else w
        ci2[w, P:P + T] = ci[p, P:P + T]
        ci2[w, P + T] = w
        tok2[w, :T] = tokens[p, :T]
        tok2[w, T] = chosen[w]
    return ci2, tok2


def key_weights(q, k, lse, scale, sees=None):
    """One (request, kv head): q [rows, group, D], k [keys, D], lse [rows, group] -> [keys]. sees[i]: how many
    keys row i sees (None: all)."""
    q, k, lse = (np.asarray(a, np.float64) for a in (q, k, lse))
    s = np.einsum("igd,jd->igj", q, k) * scale
    with np.errstate(invalid="ignore"):
        e = np.where(np.isneginf(lse)[:, :, None], 0.0, np.exp(s - np.where(np.isneginf(lse), 0.0, lse)[:, :, None]))
    if sees is not None:
        e = np.where(np.arange(k.shape[0])[None, None] < np.asarray(sees)[:, None, None], e, 0.0)
    return e.sum((0, 1))


def evict(weights, keep, sinks, recent, positions=None):
    """One (request, kv head): the slots that slots 0 .. keep - 1 hold afterwards."""
    w = np.asarray(weights, np.float64)
    n = len(w)
    keep = max(0, min(int(keep), n))
    if keep == 0:
        return np.zeros(0, np.int32)
    pos = np.arange(n) if positions is None else np.asarray(positions)
    rank = np.where(np.isnan(w), -np.inf, w + 0.0)
    nan = np.isnan(w).astype(int)
    fixed = (pos < sinks) | (pos >= pos.max() + 1 - recent)
    order = sorted(range(n), key=lambda i: (-int(fixed[i]), 0 if fixed[i] else nan[i], 0 if fixed[i] else -rank[i], i))
    live = np.zeros(n, bool)
    live[order[:keep]] = True
    source = np.arange(keep, dtype=np.int32)
    source[~live[:keep]] = keep + np.flatnonzero(live[keep:])
    return source
