"""Values near the largest number: rows whose weighted sum of |v| is finite stay finite and right."""

import numpy as np
import pytest
import torch

from paged_kv_cache_292_gb300 import binding

from chunklib import WEIGHT_ERROR, Chunks, score_error
from paritylib import assert_rounded

pytestmark = pytest.mark.gpu

LARGEST = 3.3e38


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _enlarge(b, room):
    """V of an int8 or bf16 batch times a power of two, so that no value exceeds LARGEST / room."""
    largest = 127 * float(torch.nan_to_num(b.scales[1]).max()) if b.pool == "int8" else float(torch.nan_to_num(b.cache[1]).abs().max())
    times = 2.0 ** int(torch.tensor(LARGEST / room / largest, dtype=torch.float64).log2().floor())
    held = b.scales if b.pool == "int8" else b.cache
    held[1] = (held[1].double() * times).to(held[1].dtype)
    values = torch.nan_to_num(torch.from_numpy(b.values()[1])).abs().max()
    assert LARGEST / room / 2 < float(values) <= LARGEST / room
    return b


def _decode(b, Q, **kw):
    q, k, v, ks, vs, tables, lens, _, scale = b.gpu()
    S = len(b.ctx)
    q = q.view(S, Q, b.heads, b.D) if Q > 1 else q.view(S, b.heads, b.D)
    return binding.decode_int8(q, k, v, ks, vs, tables, lens, scale, **kw).view(-1, b.heads, b.D)


@pytest.mark.parametrize("Q", [1, 2, 7])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx, num_ranges", [([20, 300, 1, 64], 1), ([20, 300, 1, 64], 0), ([5000, 33], 0)])
def test_decode_int8(Q, D, ctx, num_ranges):
    """Whole rows and merged ones.  (The sum over c tokens of weights of at most 1 times |v| is below c * max |v|.)"""
    b = Chunks([Q] * len(ctx), [max(c - Q, 0) for c in ctx], "int8", 8, 2, D, gap=0)
    _enlarge(b, int(b.ctx.max()) + 1)
    b.compare(_decode(b, Q, num_ranges=num_ranges), "large values")


@pytest.mark.parametrize("Q", [1, 3])
@pytest.mark.parametrize("times", [2.0**-60, 2.0**-90])
def test_decode_int8_of_small_values(Q, times):
    b = Chunks([Q] * 3, [40, 17, 3000], "int8", 8, 2, 128, gap=0)
    b.scales[1] *= times
    got = _decode(b, Q)
    want, spread, reach = b.want()
    b.compare((got.double() / times).to(torch.bfloat16), "small values", (want / times, spread / times, reach))


@pytest.mark.parametrize("pool", ["bf16", "int8", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [1.0, 6.0])
@pytest.mark.parametrize("new, old", [([40, 1, 300], [0, 200, 33]), ([16, 3], [3000, 5000]), ([700], [2500])])
def test_prefill(pool, D, spread, new, old):
    """Items of one and two row tiles, whole and joined; scores whose maximum moves by much (spread of K), too."""
    b = Chunks(new, old, pool, 8, 2, D, spread=spread)
    most = int(b.ctx.max()) + 1
    _enlarge(b, most)
    want, sums, reach = b.want()
    got = b.call(b.gpu())
    rows = ~np.isnan(want[:, 0, 0])
    # Weights under 2^-110 of the largest count as zero: with c tokens of at most |v| an output may miss
    # c * 2^-110 * |v|, and c * |v| is at most LARGEST.  (It shows where the tokens that weigh have code 0.)
    room = sums * (WEIGHT_ERROR[pool] + 2 * score_error(pool, D) * reach)[..., None] + LARGEST * 2.0**-110
    assert_rounded(got[torch.from_numpy(rows).cuda()], want[rows], room[rows], 1.0, "large values")


@pytest.mark.parametrize("kv_heads, D, Q", [(1, 64, 1), (1, 64, 5), (2, 128, 9)])
def test_decode_int8_as_chunks(kv_heads, D, Q):
    b = Chunks([Q] * 3, [40, 17, 3000], "int8", 4 * kv_heads, kv_heads, D, gap=0)
    _enlarge(b, int(b.ctx.max()) + 1)
    b.compare(_decode(b, Q), "large values")


@pytest.mark.parametrize("pool", ["bf16", "int8"])
@pytest.mark.parametrize("times", [2.0**-60, 2.0**-90])
def test_prefill_of_small_values(pool, times):
    b = Chunks([40, 1, 300, 20], [0, 200, 33, 3000], pool, 8, 2, 128)
    held = b.scales if pool == "int8" else b.cache
    held[1] *= times
    got = b.call(b.gpu())
    want, spread, reach = b.want()
    b.compare((got.double() / times).to(torch.bfloat16), "small values", (want / times, spread / times, reach))


@pytest.mark.parametrize("times", [3.0, 30.0])
def test_prefill_int8_of_scales_of_all_sizes(times):
    """V rows whose sizes differ by many powers of ten, in any order: a weight times its scale is rounded to 2^-8 of
    itself."""
    b = Chunks([60, 2, 300, 16], [100, 500, 40, 2000], "int8", 8, 2, 128)
    gen = torch.Generator().manual_seed(4)
    s = b.scales[1]
    s *= torch.exp(times * torch.randn(s.shape, generator=gen)).clamp(1e-25, 1e25)
    b.check("scales")
