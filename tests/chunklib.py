"""Ragged batches over paged pools for the tests of chunk attention: a batch's
inputs, the oracle's result and the bound that its outputs keep."""

from __future__ import annotations

import numpy as np
import torch

from oracle import chunks
from paged_kv_cache_292_gb300 import binding

from paritylib import assert_rounded

# Weights: bf16 (and, over int8 pools, weight times scale) half a step, 2^-8; the exponential,
# the running sums and a group's parts less than 2^-13.
WEIGHT_ERROR = {"bf16": 2.0**-8 + 2.0**-13, "int8": 2.0**-8 + 2.0**-13, "f32": 2.0**-20}


# ex2.approx.ftz gives zero for weights under 2^-126 of the largest's, so an output may miss tokens * 2^-126 * |v|
# altogether: with fewer than 2^15 tokens and |v| < 2^5, less than 2^-106.  (It shows where the tokens that weigh hold a
# zero: codes over int8 pools do.)
FLUSHED = 2.0**-106


def score_error(pool, D):
    """Error of a score (natural units) by its reach: D products summed in fp32 (tensor cores cut what does not fit, a
    whole step), and the scaling of the sum."""
    return (D + 8) * (2.0**-24 if pool == "f32" else 2.0**-23)


class Chunks:
    """Sequences of `new` tokens behind `old` others (old < 0: a context shorter than its chunk).

    Rows of the pool without a token are NaN (int8: scales NaN, codes 127), table entries without one -1, and `gap`
    rows of the token buffer lie before the first and behind the last sequence."""

    def __init__(self, new, old, pool="bf16", heads=8, kv_heads=2, D=128, bs=16, seed=0, gap=3, spread=1.0, scale=None,
                 blocks_spare=3):
        rng = np.random.default_rng([seed, 11])
        new, old = np.asarray(new), np.asarray(old)
        self.pool, self.bs, self.D, self.heads = pool, bs, D, heads
        self.ctx = (new + old).astype(np.int32)
        assert (self.ctx >= 0).all()
        self.starts = (gap + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        self.T = int(self.starts[-1]) + gap
        nblk = -(-self.ctx // bs)
        total = int(nblk.sum()) + blocks_spare
        order = rng.permutation(total)
        self.tables = np.full((len(new), int(nblk.max()) + 1), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(nblk):
            self.tables[s, :n] = order[at : at + n]
            at += n
        held = np.zeros((total, bs), dtype=bool)
        for s, c in enumerate(self.ctx):
            t = np.arange(c)
            held[self.tables[s, t // bs], t % bs] = True
        shape = (total, bs, kv_heads, D)
        x = [rng.standard_normal(shape, dtype=np.float32) for _ in range(2)]
        x[0] *= spread
        if pool == "int8":
            self.cache, self.scales = [], []
            for y in x:
                codes, scale_of = chunks.quantise(y * np.exp(0.5 * rng.standard_normal(shape[:3], dtype=np.float32))[..., None])
                codes[~held] = 127
                scale_of[~held] = np.nan
                self.cache.append(torch.from_numpy(codes))
                self.scales.append(torch.from_numpy(np.ascontiguousarray(np.swapaxes(scale_of, 1, 2))))
            self.qtype = torch.bfloat16
        else:
            self.qtype = torch.float32 if pool == "f32" else torch.bfloat16
            self.cache = []
            for y in x:
                y[~held] = np.nan
                self.cache.append(torch.from_numpy(y).to(self.qtype))
            self.scales = []
        self.q = torch.from_numpy(rng.standard_normal((self.T, heads, D), dtype=np.float32)).to(self.qtype)
        self.scale = D**-0.5 if scale is None else scale

    def values(self):
        if self.pool == "int8":
            pools = [chunks.pool_values(c.numpy(), s.numpy()) for c, s in zip(self.cache, self.scales)]
        else:
            pools = [c.double().numpy() for c in self.cache]
        return pools

    def want(self):
        k, v = (np.nan_to_num(x) for x in self.values())
        return chunks.prefill(self.q.double().numpy(), k, v, self.tables, self.ctx, self.starts, self.scale, self.bs)

    def gpu(self):
        i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
        return (self.q.cuda(), *[c.cuda() for c in self.cache], *[s.cuda() for s in self.scales], i32(self.tables),
                i32(self.ctx), i32(self.starts), self.scale)

    def call(self, args, **kw):
        return (binding.prefill_int8 if self.pool == "int8" else binding.prefill)(*args, **kw)

    def compare(self, out, what="", want=None):
        want, spread, reach = self.want() if want is None else want
        rows = ~np.isnan(want[:, 0, 0])
        room = spread * (WEIGHT_ERROR[self.pool] + 2 * score_error(self.pool, self.D) * reach)[..., None] + FLUSHED
        assert_rounded(out[torch.from_numpy(rows).to(out.device)], want[rows], room[rows], 1.0, what)
        return rows

    def check(self, what="", **kw):
        args = self.gpu()
        out = torch.full_like(args[0], 77.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert self.call(args, out=out, error_flag=err, **kw) is out
        torch.cuda.synchronize()
        assert int(err) == 0
        rows = self.compare(out, what)
        left = out[torch.from_numpy(~rows).cuda()]
        assert bool((left == 77.0).all()), "rows of no sequence were written"
        return out, args
