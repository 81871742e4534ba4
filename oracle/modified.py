"""fp64 restatement of decode with modified scores (pa_decode_mod), one query
row at a time."""

from __future__ import annotations

import numpy as np

from .paged_attention import gather_sequence


def seen_tokens(c, num_queries, i, window=0, first=0, prefix=0):
    """Bool [c]: tokens query i of num_queries sees in a sequence of c tokens."""
    pos, t = c - num_queries + i, np.arange(c)
    if pos < 0:
        return np.zeros(c, dtype=bool)
    near = (t <= pos) & ((pos - t < window) if window else True)
    return (t >= first) & (near | (t < prefix))


def seen_by_some(c, num_queries, window=0, first=0, prefix=0):
    """Bool [c]: tokens that at least one of the queries sees."""
    sees = [seen_tokens(c, num_queries, i, window, first, prefix) for i in range(num_queries)]
    return np.logical_or.reduce(sees)


def decode_mod(q, k_cache, v_cache, block_tables, context_lens, scale, block_size, *, softcap=0.0, slopes=None,
               window=0, first=None, prefix=None):
    """q [S, Q, H, D] (float64).  Returns (out, spread), both like q: ``spread`` is the same weighted sum of |v|,
    by which errors of the weights scale."""
    S, Q, H, D = q.shape
    Hk = k_cache.shape[2]
    G = H // Hk
    out, spread = np.zeros_like(q), np.zeros_like(q)
    for s in range(S):
        c = int(context_lens[s])
        mask = dict(window=window, first=int(first[s]) if first is not None else 0,
                    prefix=int(prefix[s]) if prefix is not None else 0)
        some = seen_by_some(c, Q, **mask)
        if not some.any():
            continue
        # Blocks nobody sees may have any table entry: look them up as block 0.
        row = np.array(block_tables[s], dtype=np.int64)
        hidden = np.ones(row.shape[0], dtype=bool)
        hidden[np.flatnonzero(some) // block_size] = False
        row[hidden] = 0
        k, v = gather_sequence(k_cache, row, c, block_size), gather_sequence(v_cache, row, c, block_size)
        for i in range(Q):
            t = np.flatnonzero(seen_tokens(c, Q, i, **mask))
            if t.size == 0:
                continue
            for h in range(H):
                score = scale * (k[t, h // G] @ q[s, i, h])
                if softcap:
                    score = softcap * np.tanh(score / softcap)
                if slopes is not None:
                    score = score - slopes[h] * np.abs(c - Q + i - t)
                w = np.exp(score - score.max())
                w /= w.sum()
                out[s, i, h] = w @ v[t, h // G]
                spread[s, i, h] = w @ np.abs(v[t, h // G])
    return out, spread
