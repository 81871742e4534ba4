"""The int8 cache on the GPU: codes and scales equal to the oracle's, values read back, and a run of the step's
operators together."""

import numpy as np
import pytest
import torch

from oracle import chunks
from paged_kv_cache_292_gb300 import binding

from chunklib import Chunks
from paritylib import captured

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _pools(blocks, bs, kv_heads, D, dev="cuda"):
    return [torch.full((blocks, bs, kv_heads, D), 55, dtype=torch.int8, device=dev) for _ in range(2)] + [
        torch.full((blocks, kv_heads, bs), -3.0, device=dev) for _ in range(2)]


def _write(k, v, slots, pools, **kw):
    """The pools after the GPU's write, and the oracle's."""
    want = [p.cpu().numpy().copy() for p in pools]
    binding.write_cache_int8(k.cuda(), v.cuda(), slots.cuda(), *pools, **kw)
    torch.cuda.synchronize()
    chunks.write_cache_int8(k.float().numpy(), v.float().numpy(), slots.numpy(), *want, pools[0].shape[1])
    for got, w in zip(pools, want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    return pools


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv_heads, bs, T", [(8, 16, 64), (1, 16, 1), (3, 5, 33), (2, 1, 7), (17, 24, 40), (8, 16, 3000)])
def test_codes_and_scales(dtype, D, kv_heads, bs, T):
    gen = torch.Generator().manual_seed(T + D)
    k, v = (torch.randn(T, kv_heads, D, generator=gen).mul(torch.exp(2 * torch.randn(T, kv_heads, 1, generator=gen))).to(dtype)
            for _ in range(2))
    blocks = T // bs + 3
    slots = torch.randperm(blocks * bs, generator=gen)[:T]
    slots[T // 2] = -1  # padding
    _write(k, v, slots, _pools(blocks, bs, kv_heads, D))


def test_ties_zeros_and_extremes():
    """Quotients on a tie and next to one, rows of zeros, one value, the largest and smallest magnitudes, infinities, NaN."""
    D = 128
    rows = []
    rows.append(np.concatenate([[127.0], np.arange(127) - 63.0 + 0.5]))  # scale 1: every other value a tie
    up = np.nextafter(np.float32(2.5), np.float32(3))
    rows.append(np.concatenate([[127.0], np.tile([2.5, up, np.nextafter(np.float32(2.5), np.float32(2)), -2.5, -up, 0.5, -0.5], 19)[:127]]))
    for s in (3.0, 0.7, 1e-3, 5e20):  # scales that are no powers of two: quotients all over the ties
        x = (np.arange(D) - 64 + 0.5).astype(np.float32) * np.float32(s)
        x[0] = np.float32(127 * s)
        rows.append(x)
        rows.append(np.nextafter(x, np.float32(np.inf)))
    rows.append(np.zeros(D))
    rows.append(np.where(np.arange(D) == 5, -0.0, 0.0))
    rows.append(np.where(np.arange(D) == 5, 1e-45, 0.0))  # a scale of zero: less than half a step of the smallest
    for top in (1e-44, 3e-43, 2e-42, 1e-40, 1e-38, 1.2e-36, 3.4e38):
        rows.append(np.linspace(-top, top, D))
    for bad in (np.inf, -np.inf, np.nan):
        rows.append(np.where(np.arange(D) == 77, bad, 1.0))
    x = torch.from_numpy(np.stack(rows).astype(np.float32))[:, None, :]
    slots = torch.arange(len(rows)) + 2
    _write(x, x.flip(0), slots, _pools(len(rows) // 8 + 2, 8, 1, D))
    y = x.to(torch.bfloat16)
    _write(y, y.flip(0), slots, _pools(len(rows) // 8 + 2, 8, 1, D))


def test_random_bits():
    """Any float at all."""
    rng = np.random.default_rng(5)
    bits = rng.integers(0, 2**32, (4000, 2, 64), dtype=np.uint32)
    bits[..., 1:] = (bits[..., 1:] & 0x807FFFFF) | (bits[..., :1] & 0x7F800000)  # of about one size in a row
    x = torch.from_numpy(bits.view(np.float32))
    _write(x, x.flip(0), torch.randperm(4000), _pools(500, 8, 2, 64))


def test_slots_beyond_the_pool_are_reported():
    x = torch.randn(4, 2, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _write(x, x, torch.tensor([3, 32, 2**40, -(2**40)]), _pools(4, 8, 2, 64), error_flag=err)
    assert int(err) == binding.PA_DEVERR_SLOT


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D, kv_heads, bs", [(64, 1, 16), (128, 8, 16), (128, 3, 7), (64, 20, 1)])
@pytest.mark.parametrize("firsts", [False, True])
def test_read_back(dtype, D, kv_heads, bs, firsts):
    """Rows of idle sequences, of none, in the middle of contexts; rows outside left as they were."""
    b = Chunks([70, 0, 1, 300, 0, 33], [5, 9, 0, 40, 0, 1], "int8", kv_heads, kv_heads, D, bs)
    _, k, v, ks, vs, tables, _, starts, _ = b.gpu()
    first = np.array([5, 3, 0, 40, 0, 1]) if firsts else np.zeros(6, dtype=int)
    outs = [torch.full((b.T, kv_heads, D), 9.0, dtype=dtype, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.read_cache_int8(k, v, ks, vs, tables, starts, *outs, error_flag=err,
                                  first_tokens=torch.tensor(first, dtype=torch.int32).cuda() if firsts else None)
    assert got[0] is outs[0] and int(err) == 0
    for out, values in zip(outs, b.values()):
        want = torch.full((b.T, kv_heads, D), 9.0, dtype=dtype)
        for s in range(6):
            for i in range(int(b.starts[s + 1] - b.starts[s])):
                t = int(first[s]) + i
                # code * scale in float32, rounded once more to bf16.
                row = values[b.tables[s, t // bs], t % bs].astype(np.float32)
                want[int(b.starts[s]) + i] = torch.from_numpy(row).to(dtype)
        torch.testing.assert_close(out.cpu(), want, rtol=0, atol=0)


def test_read_back_of_what_is_not_there():
    b = Chunks([20, 20], [0, 0], "int8", 2, 2, 64, 8, gap=0)
    _, k, v, ks, vs, tables, _, starts, _ = b.gpu()
    outs = [torch.full((40, 2, 64), 9.0, device="cuda") for _ in range(2)]
    for first, flag in ((2**31 - 1, binding.PA_DEVERR_CONTEXT_LEN), (-3, binding.PA_DEVERR_CONTEXT_LEN),
                        (12, binding.PA_DEVERR_BLOCK_ID)):
        for o in outs:
            o.fill_(9.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        binding.read_cache_int8(k, v, ks, vs, tables, starts, *outs, error_flag=err,
                                first_tokens=torch.tensor([first, 0], dtype=torch.int32).cuda())
        assert int(err) & flag
        plain = [torch.empty_like(o) for o in outs]
        binding.read_cache_int8(k, v, ks, vs, tables, starts, *plain)
        for o, w in zip(outs, plain):
            torch.testing.assert_close(o[20:], w[20:], rtol=0, atol=0)
            if first > 100:
                assert bool((o[:20] == 9.0).all())


def test_read_back_with_starts_that_decrease():
    """A row gets the token of a sequence that holds it, or stays as it is and is reported."""
    b = Chunks([40, 40, 40], [0, 0, 0], "int8", 2, 2, 64, 8, gap=0)
    _, k, v, ks, vs, tables, _, _, _ = b.gpu()
    starts, first = [0, 10, 5, 15], [0, 30, 2]
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = [torch.full((15, 2, 64), 9.0, device="cuda") for _ in range(2)]
    err = torch.zeros(1, **i32)
    binding.read_cache_int8(k, v, ks, vs, tables, torch.tensor(starts, **i32), *outs, error_flag=err,
                            first_tokens=torch.tensor(first, **i32))
    assert int(err) == binding.PA_DEVERR_CONTEXT_LEN
    for out, values in zip(outs, b.values()):
        for row in range(15):
            may = [np.full((2, 64), 9.0)]
            for s in range(3):
                if starts[s] <= row < starts[s + 1]:
                    t = first[s] + row - starts[s]
                    may.append(values[b.tables[s, t // 8], t % 8].astype(np.float32))
            got = out[row].cpu().numpy()
            assert any((got == m).all() for m in may), row
            assert 5 <= row < 10 or (got != 9.0).any()


def test_serving_steps_on_the_device():
    """tables_step -> write_cache_int8 -> prefill_int8 for a prompt, then decode_int8 steps in a captured graph; and the
    same prompt through read_cache_int8 and prefill over the plain rows."""
    S, Hk, H, D, bs, MB, NB = 3, 2, 8, 128, 16, 16, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    tables = torch.full((S, MB), -1, **i32)
    free, count = torch.randperm(NB, generator=gen, device="cuda").to(torch.int32), torch.tensor([NB], **i32)
    pools = [torch.zeros(NB, bs, Hk, D, dtype=torch.int8, device="cuda") for _ in range(2)] + [
        torch.full((NB, Hk, bs), float("nan"), device="cuda") for _ in range(2)]
    scale = D**-0.5
    # The prompts, with 9 rows of the token buffer to spare.
    new = torch.tensor([100, 1, 40], **i32)
    slots = torch.empty(150, dtype=torch.int64, device="cuda")
    lens, count, starts = binding.tables_step(tables, torch.zeros(S, **i32), new, free, count, bs, slots)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = rand(150, H, D), rand(150, Hk, D), rand(150, Hk, D)
    binding.write_cache_int8(k, v, slots, *pools)
    got = binding.prefill_int8(q, *pools, tables, lens, starts, scale)
    oracle_pools = lambda: [chunks.pool_values(p.cpu().numpy(), s.cpu().numpy()) for p, s in zip(pools[:2], pools[2:])]  # noqa: E731
    b = Chunks([1], [0], "int8")  # (for its bounds)
    want = chunks.prefill(q.double().cpu().numpy(), *map(np.nan_to_num, oracle_pools()), tables.cpu().numpy(),
                          lens.cpu().numpy(), starts.cpu().numpy(), scale, bs)
    b.compare(got, "prompt", want)
    # Read back into plain rows, a pool of one-token blocks; rounding them to bf16 moves scores and values by half a step.
    rows = [torch.zeros(150, Hk, D, dtype=torch.float32, device="cuda") for _ in range(2)]
    binding.read_cache_int8(*pools, tables, starts, *rows)
    own = torch.arange(150, **i32)
    one = torch.stack([torch.cat([own[int(starts[s]) : int(starts[s + 1])],
                                  torch.full((100,), -1, **i32)])[:100] for s in range(S)]).contiguous()
    plain = binding.prefill(q.float(), *[r.view(150, 1, Hk, D) for r in rows], one, lens, starts, scale)
    b2 = Chunks([1], [0], "f32")
    b2.compare(plain, "read back", want)
    # Decode steps: two graphs that swap the buffers of lengths and counts.
    q, k, v = rand(S, H, D), rand(S, Hk, D), rand(S, Hk, D)
    ones = torch.ones(S, **i32)
    slots = torch.empty(S, dtype=torch.int64, device="cuda")
    lens2, count2, starts2 = torch.empty_like(lens), torch.empty_like(count), torch.empty_like(starts)
    out = torch.empty_like(q)
    space = torch.zeros(binding.pa_decode_int8_workspace_size(S, 1, H, Hk, D), dtype=torch.uint8, device="cuda")

    def step(a, b):
        binding.tables_step(tables, a[0], ones, free, a[1], bs, slots, context_lens_out=b[0], free_count_out=b[1],
                            seq_starts=starts2)
        binding.write_cache_int8(k, v, slots, *pools)
        binding.decode_int8(q, *pools, tables, b[0], scale, out=out, workspace=space)

    graphs = [captured(lambda: step((lens, count), (lens2, count2))), captured(lambda: step((lens2, count2), (lens, count)))]
    for i in range(20):
        for x in (q, k, v):
            x.copy_(rand(*x.shape))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        now = (lens2, lens)[i % 2].cpu().numpy()
        assert list(now) == [101 + i, 2 + i, 41 + i]
        want = chunks.prefill(q.double().cpu().numpy(), *map(np.nan_to_num, oracle_pools()), tables.cpu().numpy(), now,
                              np.arange(S + 1), scale, bs)
        b.compare(out, f"step {i}", want)
