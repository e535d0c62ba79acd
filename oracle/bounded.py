"""The bounded-cache operators by definition, in double precision (numpy).

Arrays are plain numpy: caches [NB, bs, Hkv, D], q [S, H, D] as float64 values
of the 16-bit data, tables [S, MB], lens [S].  Shares no code with the CUDA
library.
"""
from __future__ import annotations

import numpy as np


def visible(n: int, window: int, sinks: int) -> list:
    """The tokens the query at the end of an n-token context sees."""
    return [j for j in range(n) if j < sinks or j >= n - window]


def rows_of(table, tokens, bs: int) -> np.ndarray:
    """Cache rows (block * bs + offset) of the given tokens."""
    return np.array([int(table[j // bs]) * bs + j % bs for j in tokens], dtype=np.int64)


def attend(q, k_cache, v_cache, tables, lens, scale, window=None, sinks=0):
    """(out [S, H, D], weights, magnitude [S, H, D]): weights[s] is (tokens,
    [H, len(tokens)]); magnitude = sum_j p_j |V_j|, for error bounds."""
    S, H, D = q.shape
    bs, Hkv = k_cache.shape[1], k_cache.shape[2]
    G = H // Hkv
    k_rows, v_rows = k_cache.reshape(-1, Hkv, D), v_cache.reshape(-1, Hkv, D)
    out, mag, weights = np.zeros((S, H, D)), np.zeros((S, H, D)), []
    for s in range(S):
        n = int(lens[s])
        tok = list(range(n)) if window is None else visible(n, window, sinks)
        r = rows_of(tables[s], tok, bs)
        p = np.zeros((H, len(tok)))
        for h in range(H):
            if not tok:
                continue
            z = scale * (k_rows[r, h // G] @ q[s, h])
            w = np.exp(z - z.max())
            p[h] = w / w.sum()
            out[s, h] = p[h] @ v_rows[r, h // G]
            mag[s, h] = p[h] @ np.abs(v_rows[r, h // G])
        weights.append((tok, p))
    return out, weights, mag


def accumulate(scores, weights, Hkv: int) -> np.ndarray:
    """scores [S, Hkv, cap] (float64 copy) plus each token's weight."""
    out = np.array(scores, dtype=np.float64)
    for s, (tok, p) in enumerate(weights):
        G = p.shape[0] // Hkv
        for g in range(Hkv):
            for h in range(g * G, (g + 1) * G):
                out[s, g, tok] += p[h]
    return out


def evict_row(score, stored, n: int, seen: int, budget: int, recent: int, sinks: int):
    """One (sequence, head): returns (source, position): entry i < budget
    takes what entry source[i] held, whose position is position[i]; None when
    nothing is evicted.  Kept: protected tokens, then falling score, ties by
    the lowest index; NaN as -inf."""
    if n <= budget:
        return None
    pos = [int(stored[j]) if stored[j] >= 0 else seen - n + j for j in range(n)]

    def rank(j):
        v = float(score[j])
        safe = pos[j] < sinks or pos[j] >= seen - recent
        return (0 if safe else 1, 0.0 if safe else -(-np.inf if np.isnan(v) else v), j)

    kept = set(sorted(range(n), key=rank)[:budget])
    movers = [j for j in range(budget, n) if j in kept]
    source = []
    for i in range(budget):
        source.append(i if i in kept else movers.pop(0))
    assert not movers
    return source, [pos[j] for j in source]


def evict(k_cache, v_cache, scores, positions, tables, lens, seen, budget, recent, sinks):
    """In place on numpy copies of any dtype; returns the new lengths."""
    bs, Hkv, D = k_cache.shape[1:]
    k_rows, v_rows = k_cache.reshape(-1, Hkv, D), v_cache.reshape(-1, Hkv, D)
    for s in range(len(lens)):
        n = int(lens[s])
        for g in range(Hkv):
            r = evict_row(scores[s, g], positions[s, g], n, int(seen[s]), budget, recent, sinks)
            if r is None:
                continue
            source, pos = r
            to = rows_of(tables[s], range(budget), bs)
            of = rows_of(tables[s], source, bs)
            k_rows[to, g] = k_rows[of, g].copy()
            v_rows[to, g] = v_rows[of, g].copy()
            scores[s, g, :budget] = scores[s, g, source].copy()
            scores[s, g, budget:n] = 0
            positions[s, g, :budget] = pos
            positions[s, g, budget:n] = -1
    return np.minimum(np.asarray(lens), budget)
