"""Decode over int8 pools: forced ranges, scales of very different sizes, tokens whose scale is NaN, workspaces."""

import numpy as np
import pytest
import torch

from paged_kv_cache_292_gb300 import binding

from chunklib import Chunks
from paritylib import assert_rounded, captured, refused_under_capture

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _batch(ctx, Q=1, heads=8, kv_heads=2, D=128, bs=16, **kw):
    return Chunks([Q] * len(ctx), [c - Q for c in ctx], "int8", heads, kv_heads, D, bs, gap=0, **kw)


def _call(b, Q, **kw):
    q, k, v, ks, vs, tables, lens, _, scale = b.gpu()
    S = len(b.ctx)
    q = q.view(S, Q, b.heads, b.D) if Q > 1 else q.view(S, b.heads, b.D)
    return binding.decode_int8(q, k, v, ks, vs, tables, lens, scale, **kw).view(-1, b.heads, b.D)


@pytest.mark.parametrize("num_ranges", [1, 2, 7, 152, 400])
@pytest.mark.parametrize("Q", [1, 2, 4])
def test_ranges(num_ranges, Q):
    b = _batch([700, 1, 0, 33, 2000, 16], Q)
    b.compare(_call(b, Q, num_ranges=num_ranges), f"{num_ranges} ranges")


@pytest.mark.parametrize("D, kv_heads, group", [(64, 2, 1), (64, 8, 4), (128, 1, 8), (128, 8, 4), (128, 3, 5), (64, 1, 4), (128, 16, 2)])
@pytest.mark.parametrize("Q", [1, 2, 7])
@pytest.mark.parametrize("bs", [16, 8, 4, 6, 1])
def test_shapes(D, kv_heads, group, Q, bs):
    b = _batch([130, 17, 2, 64], Q, kv_heads * group, kv_heads, D, bs)
    b.compare(_call(b, Q), "shapes")


@pytest.mark.parametrize("Q", [1, 2])
@pytest.mark.parametrize("spread", [3.0, 30.0])
def test_scales_of_all_sizes(Q, spread):
    """V rows whose sizes differ by many powers of ten, in any order: a weight times its scale is rounded to 2^-11 of
    itself, or to 2^-38 of the largest weight times the largest scale (of 127 codes and c tokens)."""
    ctx = [500, 90, 16, 300]
    b = _batch(ctx, Q)
    rng = np.random.default_rng(4)
    s = b.scales[1]
    s *= torch.from_numpy(np.exp(spread * rng.standard_normal(tuple(s.shape))).astype(np.float32)).clamp(1e-30, 1e30)
    want, spread_of, reach = b.want()
    room = spread_of * (2.0**-8 + 2.0**-13 + 2 * (b.D + 8) * 2.0**-23 * reach[..., None])
    for i, c in enumerate(ctx):
        held = s.numpy()[b.tables[i, np.arange(c) // b.bs], :, np.arange(c) % b.bs]
        room[i * Q : (i + 1) * Q] += 2.0**-38 * held.max() * 127 * c
    assert_rounded(_call(b, Q), want, room, 1.0, "scales")


@pytest.mark.parametrize("Q", [2, 4])
def test_nan_scales_reach_only_queries_that_see_them(Q):
    b = _batch([100, 300], Q)
    for pool in (0, 1):
        t = 300 - Q + 1  # seen by all queries of sequence 1 but the first
        block, row = b.tables[1, t // 16], t % 16
        keep = b.scales[pool][block, 1, row].clone()
        b.scales[pool][block, 1, row] = float("nan")
        out = _call(b, Q).view(2, Q, 8, 128)
        b.scales[pool][block, 1, row] = keep
        assert bool(torch.isnan(out[1, 1:, 4:]).all())
        rest = torch.isfinite(out)
        assert bool(rest[0].all()) and bool(rest[1, 0].all()) and bool(rest[1, :, :4].all())


def test_zero_rows_and_largest_codes():
    """Keys and values of zero scale; rows all at +-127."""
    b = _batch([40, 200])
    for pool in (0, 1):
        b.scales[pool][:, :, ::3] = 0.0
        b.cache[pool][:, 1::3] = torch.where(torch.rand(b.cache[pool][:, 1::3].shape) < 0.5, -127, 127).to(torch.int8)
    # (rows without a token stay NaN)
    held = np.zeros(b.scales[0].shape, dtype=bool)
    for s, c in enumerate(b.ctx):
        t = np.arange(c)
        held[b.tables[s, t // 16], :, t % 16] = True
    for pool in (0, 1):
        b.scales[pool][torch.from_numpy(~held)] = float("nan")
    b.compare(_call(b, 1), "zeros")
    for pool in (0, 1):
        b.scales[pool][torch.from_numpy(held)] = 0.0
    out = _call(b, 1)
    assert bool((out == 0).all())


@pytest.mark.parametrize("Q, kv_heads, D", [(1, 2, 128), (3, 2, 128), (1, 1, 64), (9, 1, 128)])
def test_workspaces_and_capture(Q, kv_heads, D):
    """A workspace shared by shapes of both kinds stays fit for the decode kernel's tickets."""
    b, other = _batch([900, 20, 3000], Q, 4 * kv_heads, kv_heads, D), _batch([2000, 70, 500], 1)
    size = max(binding.pa_decode_int8_workspace_size(3, Q, 4 * kv_heads, kv_heads, D),
               binding.pa_decode_int8_workspace_size(3, 1, 8, 2, 128))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        b.compare(_call(b, Q, workspace=ws), "first")
        other.compare(_call(other, 1, workspace=ws), "second")
    small = binding.pa_decode_int8_workspace_size(3, Q, 4 * kv_heads, kv_heads, D)
    with pytest.raises(binding.PagedAttnError) as e:
        _call(b, Q, workspace=ws[: small - 256])
    assert e.value.code == binding.PA_ERR_WORKSPACE
    q, k, v, ks, vs, tables, lens, _, scale = b.gpu()
    q = q.view(3, Q, 4 * kv_heads, D)
    out = torch.empty_like(q)
    assert refused_under_capture(lambda: binding.decode_int8(q, k, v, ks, vs, tables, lens, scale, out=out),
                                 binding.PagedAttnError)
    own = torch.zeros(small, dtype=torch.uint8, device="cuda")
    graph = captured(lambda: binding.decode_int8(q, k, v, ks, vs, tables, lens, scale, out=out, workspace=own))
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        b.compare(out.view(-1, 4 * kv_heads, D), "replay")


def test_refusals_of_the_python_layer():
    b = _batch([40, 20])
    q, k, v, ks, vs, tables, lens, starts, scale = b.gpu()
    good = (q, k, v, ks, vs, tables, lens, scale)
    binding.decode_int8(*good)

    def refused(call, *args, **kw):
        with pytest.raises(ValueError):
            call(*args, **kw)

    for i, bad in ((0, q.float()), (0, q.transpose(0, 1)), (1, k.to(torch.uint8)), (1, k.transpose(1, 2)), (2, v[:1]),
                   (3, ks.transpose(1, 2)), (3, ks.double()), (4, vs[:1]), (5, tables.long()), (6, lens[:1]), (5, tables.cpu()),
                   (3, ks.cpu())):
        args = list(good)
        args[i] = bad
        refused(binding.decode_int8, *args)
    refused(binding.decode_int8, *good, out=q[:1])
    chunk = (q, k, v, ks, vs, tables, lens, starts, scale)
    binding.prefill_int8(*chunk)
    refused(binding.prefill_int8, *chunk[:7], starts[:-1], scale)
    refused(binding.prefill_int8, *chunk[:7], starts.long(), scale)
    refused(binding.prefill, q, k, v, tables, lens, starts, scale)  # int8 pools want their scales
    refused(binding.prefill, q.float(), k.bfloat16(), v.bfloat16(), tables, lens, starts, scale)
    refused(binding.prefill, q, k.bfloat16(), v.bfloat16(), tables, lens[:1], starts, scale)
    refused(binding.prefill, q, k.bfloat16(), v.bfloat16(), tables, lens, starts, scale, out=q[:1])
    rows, slots = torch.zeros(3, 2, 128, device="cuda"), torch.arange(3, device="cuda")
    binding.write_cache_int8(rows, rows, slots, k, v, ks, vs)
    refused(binding.write_cache_int8, rows, rows.bfloat16(), slots, k, v, ks, vs)
    refused(binding.write_cache_int8, rows, rows, slots.int(), k, v, ks, vs)
    refused(binding.write_cache_int8, rows, rows[:2], slots, k, v, ks, vs)
    refused(binding.write_cache_int8, rows.half(), rows.half(), slots, k, v, ks, vs)
    out = torch.zeros(2, 2, 128, device="cuda")
    binding.read_cache_int8(k, v, ks, vs, tables, starts, out, out.clone())
    refused(binding.read_cache_int8, k, v, ks, vs, tables, starts, out, out.bfloat16())
    refused(binding.read_cache_int8, k, v, ks, vs, tables, starts[:-1], out, out)
    refused(binding.read_cache_int8, k, v, ks, vs, tables, starts, out, out, first_tokens=starts)
    refused(binding.read_cache_int8, k, v, ks, vs, tables, starts, out[:, :1], out)


def test_odd_starts_stay_inside():
    """Starts that decrease, leave the buffer or skip rows: reported, and the sequences with good ones are right."""
    b = Chunks([20, 30, 140], [100, 40, 20], "bf16", 4, 2, 64, 16)
    want = b.want()
    args = list(b.gpu())
    for starts, good in (([3, 23, 10, 193], [0]), ([-50, 23, 53, 193], [1, 2]), ([3, 23, 53, 10**9], [0, 1]),
                         ([-(2**31), 2**31 - 1, 53, 193], [2])):
        args[-2] = torch.tensor(starts, dtype=torch.int32).cuda()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = binding.prefill(*args, error_flag=err)
        torch.cuda.synchronize()
        assert int(err) & binding.PA_DEVERR_CONTEXT_LEN
        rows = np.zeros(b.T, dtype=bool)
        for s in good:
            rows[int(b.starts[s]) : int(b.starts[s + 1])] = True
        if starts[2] == 10:
            rows[10:] = False  # two sequences claim these
        if starts[1] > 2**30:
            rows[:] = False
            rows[53:193] = False
        keep = [np.where(rows.reshape(-1, *[1] * (x.ndim - 1)), x, np.nan) for x in want]
        if rows.any():
            b.compare(out, str(starts), keep)
