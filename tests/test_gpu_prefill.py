"""GPU parity of chunk attention (pa_prefill, pa_prefill_int8, pa_decode_int8) against the fp64 restatement."""

import numpy as np
import pytest
import torch

from paged_kv_cache_292_gb300 import binding

from chunklib import Chunks
from paritylib import captured, refused_under_capture

pytestmark = pytest.mark.gpu

POOLS = ["bf16", "int8", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


@pytest.mark.parametrize("pool", POOLS)
def test_one_token(pool):
    Chunks([1], [0], pool, heads=1, kv_heads=1).check("v itself")


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (8, 2), (3, 3), (14, 2), (8, 1), (12, 4), (5, 1), (6, 1)])
def test_heads(pool, D, heads, kv_heads):
    Chunks([70, 1, 9, 0, 130], [30, 200, 0, 50, 7], pool, heads, kv_heads, D).check("heads")


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("old", [0, 1, 127, 128, 300])
def test_lengths(pool, n, old):
    """Chunks around one and two row tiles, contexts around one and two tiles of tokens (group 2)."""
    Chunks([n], [old], pool, 4, 2, 64).check(f"{n} on {old}")


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("bs", [1, 2, 3, 4, 5, 7, 8, 12, 16, 24, 40, 100, 128, 256])
def test_block_sizes(pool, bs):
    Chunks([40, 3, 150], [100, 5, 130], pool, 4, 2, 128 if bs % 3 else 64, bs).check(f"bs={bs}")


@pytest.mark.parametrize("pool", POOLS)
def test_contexts_shorter_than_the_chunk(pool):
    """Rows whose position is negative are zero; a context of no token at all; idle sequences around them."""
    out, _ = Chunks([5, 300, 0, 200, 1, 0], [-5, -300, 0, -170, -1, 40], pool, 4, 1, 64).check("short")
    assert bool((out[3:8] == 0).all())


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("n, old", [(1, 20000), (3, 9000), (16, 9000), (40, 5000), (300, 4000)])
def test_divided_contexts(pool, n, old):
    """Few rows on a long context: the list's ranges cut the one item of a head many times."""
    Chunks([n], [old], pool, 4, 1).check("divided")


@pytest.mark.parametrize("pool", POOLS)
def test_many_sequences(pool):
    """More sequences than threads of a CTA, of every kind."""
    rng = np.random.default_rng(3)
    new = np.where(rng.random(700) < 0.8, 1, rng.integers(0, 40, 700))
    Chunks(new, rng.integers(0, 90, 700), pool, 2, 1, 64, 8).check("many")


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("seed", range(6))
def test_random_batches(pool, seed):
    rng = np.random.default_rng([seed, 8])
    S, kv = int(rng.integers(1, 9)), int(rng.integers(1, 4))
    new = rng.integers(0, 260, S)
    new[rng.integers(0, S)] += 1
    old = np.maximum(rng.integers(-20, 700, S), -new)
    Chunks(new, old, pool, kv * int(rng.integers(1, 9)), kv, int(rng.choice([64, 128])), int(rng.choice([8, 16, 17, 32])),
           seed).check("random")


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_scales_and_strong_scores(pool, scale):
    Chunks([80, 2], [100, 300], pool, 4, 2, 64, scale=scale, spread=3.0).check("scale")


@pytest.mark.parametrize("pool", POOLS)
def test_same_bits_again(pool):
    """No order of additions depends on timing."""
    b = Chunks([300, 1, 40], [1500, 3000, 0], pool, 8, 2)
    args = b.gpu()
    first = b.call(args)
    for _ in range(3):
        torch.testing.assert_close(b.call(args)[3:-3], first[3:-3], rtol=0, atol=0)


@pytest.mark.parametrize("D, Q, heads, kv_heads", [(128, 1, 8, 2), (64, 1, 8, 1), (128, 3, 8, 2), (128, 40, 4, 4)])
def test_decode_int8(D, Q, heads, kv_heads):
    """The same number of queries for every sequence, with empty rows and contexts shorter than the queries."""
    ctx = [300, 17, 1, 0, 1000, 2]
    b = Chunks([Q] * len(ctx), [c - Q for c in ctx], "int8", heads, kv_heads, D, gap=0)
    q, k, v, ks, vs, tables, lens, _, scale = b.gpu()
    q = q.view(len(ctx), Q, heads, D) if Q > 1 else q.view(len(ctx), heads, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.decode_int8(q, k, v, ks, vs, tables, lens, scale, error_flag=err)
    assert out.shape == q.shape and int(err) == 0
    b.compare(out.view(-1, heads, D), "decode")


def test_int8_nan_scales_reach_only_rows_that_see_them():
    b = Chunks([200], [100], "int8", 4, 2, 128, 16, gap=0)
    _, clean_v = b.values()
    for pool in (0, 1):
        block, row = b.tables[0, 250 // 16], 250 % 16
        keep = b.scales[pool][block, 1, row].clone()
        b.scales[pool][block, 1, row] = float("nan")
        out = b.call(b.gpu())
        b.scales[pool][block, 1, row] = keep
        assert bool(torch.isnan(out[150:, 2:]).all()) and bool(torch.isfinite(out[:150]).all())
        assert bool(torch.isfinite(out[150:, :2]).all())
    del clean_v


@pytest.mark.parametrize("pool", POOLS)
def test_capture_streams_and_workspace(pool):
    b, other = Chunks([300, 1, 20], [700, 4000, 0], pool, 8, 2), Chunks([33], [3000], pool, 8, 2, seed=5)
    args, args2 = b.gpu(), other.gpu()
    size = binding.pa_prefill_workspace_size(b.D)
    spaces = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(args[0]), torch.empty_like(args2[0])]
    b.call(args, out=outs[0], workspace=spaces[0])
    torch.cuda.synchronize()
    b.compare(outs[0], "caller's workspace")
    assert refused_under_capture(lambda: b.call(args, out=outs[0]), binding.PagedAttnError)
    graphs = [captured(lambda: b.call(args, out=outs[0], workspace=spaces[0])),
              captured(lambda: other.call(args2, out=outs[1], workspace=spaces[1]))]
    for _ in range(2):
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        b.compare(outs[0], "replay")
        other.compare(outs[1], "replay")
    # Two streams at once, each with the library's own buffer.
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got = [x.call(a, stream=s) for x, a, s in ((b, args, streams[0]), (other, args2, streams[1]))]
    torch.cuda.synchronize()
    b.compare(got[0], "stream 0")
    other.compare(got[1], "stream 1")
    with pytest.raises(binding.PagedAttnError) as e:
        b.call(args, workspace=spaces[0][: size - 1])
    assert e.value.code == binding.PA_ERR_WORKSPACE


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("bs", [16, 5])
def test_bad_inputs_are_reported(pool, bs):
    """Bad block ids, lengths and starts: reported, nothing else harmed."""
    b = Chunks([20, 30, 140], [100, 40, 20], pool, 4, 2, 64, bs)
    clean = b.want()
    for bad in (10**6, -7):
        args = list(b.gpu())
        tables = args[-4].clone()
        tables[1, 2] = bad
        args[-4] = tables
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = b.call(args, error_flag=err)
        assert int(err) == binding.PA_DEVERR_BLOCK_ID
        keep = [np.where((np.arange(b.T) >= b.starts[1]) & (np.arange(b.T) < b.starts[2])[None] if x.ndim == 1 else
                         ((np.arange(b.T) >= b.starts[1]) & (np.arange(b.T) < b.starts[2])).reshape(-1, *[1] * (x.ndim - 1)),
                         np.nan, x) for x in clean]
        b.compare(out, "bad block", keep)
    for where, value in ((-3, 10**6), (-3, -4), (-2, 10**6)):
        args = list(b.gpu())
        x = args[where].clone()
        x[2 if where == -3 else 3] = value
        args[where] = x
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if where == -3 and value > 0:  # lengths are clamped to the row, whose last entries are no blocks
            tables = args[-4].clone()
            tables[2, tables[2] < 0] = 0
            args[-4] = tables
        out = b.call(args, error_flag=err)
        assert int(err) & binding.PA_DEVERR_CONTEXT_LEN
        rows = np.arange(b.T) < b.starts[2]
        keep = [np.where(rows.reshape(-1, *[1] * (x.ndim - 1)), x, np.nan) for x in clean]
        b.compare(out, "bad length", keep)


def test_no_tokens():
    b = Chunks([1], [3], "bf16", 4, 2, gap=0)
    q, k, v, tables, lens, starts, scale = b.gpu()
    assert binding.prefill(q[:0], k, v, tables, lens, torch.zeros_like(starts), scale).shape == (0, 4, 128)
    out = torch.full_like(q, 5.0)
    binding.prefill(q, k, v, tables, lens, torch.zeros_like(starts), scale, out=out)
    assert bool((out == 5.0).all())
