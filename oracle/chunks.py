"""fp64 restatement of chunk attention (pa_prefill) and of the int8 cache, one
sequence and one head at a time."""

from __future__ import annotations

import numpy as np

from .paged_attention import gather_sequence


def prefill(q, k_cache, v_cache, block_tables, context_lens, seq_starts, scale, block_size):
    """q [T, H, D] (float64).  Returns (out, spread, reach), NaN in rows of no sequence.  ``spread`` [T, H, D] is the
    same weighted sum of |v|, by which relative errors of the weights scale, and ``reach`` [T, H] the largest
    |scale| * sum |q k|, by which rounded scores do."""
    T, H, D = q.shape
    G = H // k_cache.shape[2]
    out, spread, reach = np.full_like(q, np.nan), np.full_like(q, np.nan), np.full((T, H), np.nan)
    for s in range(len(context_lens)):
        a, b, c = int(seq_starts[s]), int(seq_starts[s + 1]), int(context_lens[s])
        if a == b:
            continue
        out[a:b] = spread[a:b] = reach[a:b] = 0.0
        k = gather_sequence(k_cache, np.asarray(block_tables[s]), c, block_size)
        v = gather_sequence(v_cache, np.asarray(block_tables[s]), c, block_size)
        pos = c - (b - a) + np.arange(b - a)
        rows = np.flatnonzero(pos >= 0)
        if rows.size == 0:
            continue
        hidden = np.arange(c)[None, :] > pos[rows, None]
        for h in range(H):
            x = q[a + rows, h]
            score = np.where(hidden, -np.inf, scale * (x @ k[:, h // G].T))
            w = np.exp(score - score.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[a + rows, h] = w @ v[:, h // G]
            spread[a + rows, h] = w @ np.abs(v[:, h // G])
            reach[a + rows, h] = np.where(hidden, 0.0, abs(scale) * (np.abs(x) @ np.abs(k[:, h // G]).T)).max(1)
    return out, spread, reach


def quantise(x):
    """(codes int8, scales float32) of rows x [..., D] (float32 or narrower): scale = max |x| / 127 in float32, codes
    the nearest integers of the exact x / scale, ties to even.  (The quotient of two float32 numbers that is not on
    a tie is further from it than float64 rounds.)  A row that is not finite: codes 0, scale NaN."""
    x = np.asarray(x, dtype=np.float32)
    finite = np.isfinite(x).all(-1)
    safe = np.where(finite[..., None], x, 0).astype(np.float32)
    scale = (np.abs(safe).max(-1) / np.float32(127)).astype(np.float32)
    steps = safe.astype(np.float64) / np.where(scale > 0, scale, 1).astype(np.float64)[..., None]
    codes = np.clip(np.rint(np.where(scale[..., None] > 0, steps, 0.0)), -127, 127).astype(np.int8)
    return codes, np.where(finite, scale, np.float32(np.nan)).astype(np.float32)


def values(codes, scales):
    """float64 values of codes [..., D] by their rows' scales."""
    return np.asarray(codes, dtype=np.float64) * np.asarray(scales, dtype=np.float64)[..., None]


def write_cache_int8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scales, v_scales, block_size):
    """In place: the rows' codes and scales at their slots (negative slots and those beyond the pool skipped)."""
    for new, pool, scales in ((k_new, k_cache, k_scales), (v_new, v_cache, v_scales)):
        codes, scale = quantise(new)
        for i, slot in enumerate(np.asarray(slot_mapping)):
            if 0 <= slot < pool.shape[0] * block_size:
                pool[slot // block_size, slot % block_size] = codes[i]
                scales[slot // block_size, :, slot % block_size] = scale[i]


def pool_values(pool, scales):
    """float64 [NB, bs, Hk, D] of an int8 pool with scales [NB, Hk, bs]."""
    return values(pool, np.swapaxes(scales, 1, 2))
