"""Oracle: attention over packed sequences, over a prefix shared by a batch next to caches of
its own, the append to such caches and the eviction from them, in float64 (test
infrastructure only).

What is computed, row by row from the definitions (the pages describe one sequence per call
and have no counterpart):

* packed: query i of a sequence with Lq queries and Lk keys sees key c when c < Lk and, with
  the causal mask, c <= i + Lk - Lq;
* shared prefix: query token t of T sees every prefix key, and key c of its sequence's own
  cache when c <= n - T + t (n live entries, the T new ones included);
* softmax with the caller's float32 scale taken exactly; a row that sees no key has O = 0 and
  LSE = -inf; query head h reads key/value head h // (Hq // Hkv);
* weight: each own cache key collects its attention probability over all query rows;
* append: T rows at the place of a sequence's length, weight 0;
* eviction: of n > budget entries the first ``sinks``, the last ``recent`` and, of the rest,
  those of largest weight stay (ties: the lower index; NaN ranks below every number), in
  their order.

Inputs arrive as bf16-valued arrays; they are widened to float64 exactly.
"""
from __future__ import annotations

import numpy as np

from .attention import _as_f64


def _rows(q, keys, values, seen, scale):
    """One head: q [n, d], keys/values [m, d], seen bool [n, m] -> O, LSE, P, sum P |v|."""
    s = scale * (q @ keys.T) if keys.shape[0] else np.zeros((q.shape[0], 0))
    s = np.where(seen, s, -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    e = np.where(seen, np.exp(s - np.where(np.isneginf(m), 0.0, m)[:, None]), 0.0)
    l = e.sum(axis=1)
    some = seen.any(axis=1)
    p = e / np.where(some, l, 1.0)[:, None]
    # unseen keys take no part, whatever their values are
    used = seen.any(axis=0)
    o = p[:, used] @ values[used]
    mag = p[:, used] @ np.abs(values[used])
    with np.errstate(divide="ignore"):
        lse = np.where(some, m + np.log(np.where(some, l, 1.0)), -np.inf)
    return o, lse, p, mag


def packed_attention(q, k, v, cu_q, cu_k, scale: float, causal: bool):
    """q [Tq, Hq, d], k, v [Tk, Hkv, d] -> O [Tq, Hq, d], LSE [Hq, Tq] and sum_c p |v|
    [Tq, Hq, d] (the scale of O's rounding); rows in no sequence stay NaN."""
    q, k, v = _as_f64(q), _as_f64(k), _as_f64(v)
    sc = float(np.float32(scale))
    hq, hk = q.shape[1], k.shape[1]
    o, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full((hq, q.shape[0]), np.nan)
    for s in range(len(cu_q) - 1):
        a, b, ka, kb = int(cu_q[s]), int(cu_q[s + 1]), int(cu_k[s]), int(cu_k[s + 1])
        n, m = b - a, kb - ka
        i, c = np.arange(n)[:, None], np.arange(m)[None, :]
        seen = (c <= i + m - n) if causal else np.ones((n, m), dtype=bool)
        for h in range(hq):
            g = h // (hq // hk)
            o[a:b, h], lse[h, a:b], _, mag[a:b, h] = _rows(q[a:b, h], k[ka:kb, g], v[ka:kb, g], seen, sc)
    return o, lse, mag


def shared_prefix_attention(q, prefix_k, prefix_v, k_cache, v_cache, lens, scale: float):
    """q [B, T, Hq, d], prefix [Lp, Hkv, d], caches [B, Hkv, cap, d], lens [B] -> O like q, LSE
    [B, Hq, T], sum p |v| like q, and the weight [B, Hkv, cap] that each cache key collects."""
    q, prefix_k, prefix_v = _as_f64(q), _as_f64(prefix_k), _as_f64(prefix_v)
    k_cache, v_cache = _as_f64(k_cache), _as_f64(v_cache)
    sc = float(np.float32(scale))
    B, T, hq, d = q.shape
    hk, cap = k_cache.shape[1], k_cache.shape[2]
    lp = prefix_k.shape[0]
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, weight = np.zeros((B, hq, T)), np.zeros((B, hk, cap))
    for b in range(B):
        n = int(lens[b])
        t, c = np.arange(T)[:, None], np.arange(n)[None, :]
        seen = np.concatenate([np.ones((T, lp), dtype=bool), c <= n - T + t], axis=1)
        for h in range(hq):
            g = h // (hq // hk)
            keys = np.concatenate([prefix_k[:, g], k_cache[b, g, :n]])
            values = np.concatenate([prefix_v[:, g], v_cache[b, g, :n]])
            o[b, :, h], lse[b, h], p, mag[b, :, h] = _rows(q[b, :, h], keys, values, seen, sc)
            weight[b, g, :n] += p[:, lp:].sum(axis=0)
    return o, lse, mag, weight


def evict_kept(weight, n: int, budget: int, sinks: int, recent: int):
    """Indices that stay, ascending, of one head's n entries."""
    if n <= budget:
        return np.arange(n)
    middle = np.arange(sinks, n - recent)
    w = np.asarray(weight, dtype=np.float64)[middle]
    # rank: numbers by falling weight, NaN last, ties by index
    order = sorted(range(len(middle)), key=lambda j: (bool(np.isnan(w[j])), 0.0 if np.isnan(w[j]) else -w[j], j))
    chosen = middle[sorted(order[:budget - sinks - recent])]
    return np.concatenate([np.arange(sinks), chosen, np.arange(n - recent, n)])
