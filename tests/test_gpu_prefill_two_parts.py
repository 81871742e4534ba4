"""Items of one row tile carry the softmax weights in two bf16 parts.  Half of the tokens have a weight that lies next to
the middle between two bf16 numbers, and V cancels the two halves, so that the roundings of one part alone add up."""

import numpy as np
import pytest
import torch

from oracle import chunks

from chunklib import Chunks, score_error
from paritylib import assert_rounded

# Two parts: half a step of bf16, twice, 2^-16.  The exponential, the running sums and a group's parts less than 2^-13.
WEIGHT_ERROR = 2.0**-16 + 2.0**-13


def _bf16(x):
    return torch.as_tensor(x, dtype=torch.float64).to(torch.bfloat16).double().numpy()


def _score():
    """The bf16 score below zero whose weight is farthest, by its size, from a bf16 number."""
    s = np.unique(_bf16(-np.linspace(0.1, 1.0, 4000)))
    w = np.exp(s)
    return float(s[np.argmax(np.abs(_bf16(w) - w) / w)])


def _batch(pool, new, old, heads, kv_heads, D, bs=16):
    """Even tokens: weight 1, V near exp(score); odd ones: weight exp(score), V -1.  One dim of the queries is not zero."""
    b = Chunks(new, old, pool, heads, kv_heads, D, bs, scale=1.0)
    score = _score()
    value = float(_bf16(np.exp(score)))
    b.q.zero_()
    b.q[..., 0] = 1.0
    for s, c in enumerate(b.ctx):
        t = np.arange(c)
        block, row, odd = b.tables[s, t // b.bs], t % b.bs, torch.from_numpy(t % 2 == 1)
        k, v = torch.where(odd, score, 0.0), torch.where(odd, -1.0, value)
        for x, rows in ((0, k[:, None, None].expand(-1, kv_heads, D)), (1, v[:, None, None].expand(-1, kv_heads, D))):
            if pool == "int8":
                b.cache[x][block, row] = 64
                b.scales[x][block, :, row] = (rows[..., 0] / 64).float()
            else:
                b.cache[x][block, row] = rows.to(b.cache[x].dtype)
    return b


def _room(b):
    want, spread, reach = b.want()
    rows = ~np.isnan(want[:, 0, 0])
    return want[rows], spread[rows] * (WEIGHT_ERROR + 2 * score_error(b.pool, b.D) * reach[rows])[..., None], rows


SHAPES = [([1, 16, 32], [2000, 900, 64], 8, 2, 128), ([16, 5], [700, 3000], 16, 2, 64), ([128, 100], [300, 0], 2, 2, 128),
          ([42, 1], [500, 90], 6, 2, 64)]


@pytest.mark.parametrize("pool", ["bf16", "int8"])
@pytest.mark.parametrize("new, old, heads, kv_heads, D", SHAPES)
def test_one_part_would_show(pool, new, old, heads, kv_heads, D):
    """The bound is tight enough: weights (over int8 pools, weights times V's scales) in one bf16 part break it."""
    b = _batch(pool, new, old, heads, kv_heads, D)
    want, room, rows = _room(b)
    score, value = _score(), float(_bf16(np.exp(_score())))
    seen = np.concatenate([np.arange(c - n + 1, c + 1) for n, c in zip(new, b.ctx)])
    even, odd = (seen + 1) // 2, seen // 2
    w = np.exp(score)
    out = (even * value - odd * _bf16(w)) / (even + odd * w)
    exact = (even * value - odd * w) / (even + odd * w)
    np.testing.assert_allclose(want, np.broadcast_to(exact[:, None, None], want.shape), atol=1e-12)
    over = np.abs(out - exact)[:, None, None] - 2.0**-8 * np.abs(want) - room
    assert over[seen > 60].min() > 0


@pytest.mark.gpu
@pytest.mark.parametrize("pool", ["bf16", "int8"])
@pytest.mark.parametrize("new, old, heads, kv_heads, D", SHAPES)
@pytest.mark.parametrize("bs", [16, 5])
def test_two_parts(pool, new, old, heads, kv_heads, D, bs):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import binding, build

    build.build()
    binding.load()
    b = _batch(pool, new, old, heads, kv_heads, D, bs)
    want, room, rows = _room(b)
    got = b.call(b.gpu())
    assert_rounded(got[torch.from_numpy(rows).cuda()], want, room, 1.0, "two parts")


def test_the_oracle_reads_the_pools_as_made():
    b = _batch("int8", [3], [4], 2, 1, 64)
    k, v = (chunks.pool_values(c.numpy(), s.numpy()) for c, s in zip(b.cache, b.scales))
    t = np.arange(7)
    at = (b.tables[0, t // 16], t % 16)
    assert np.allclose(k[at][:, 0, 0], np.where(t % 2, _score(), 0.0)) and np.allclose(v[at][1::2], -1.0)
