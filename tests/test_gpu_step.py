"""Serving steps on the device: tables and slots from lengths, cache write, decode
over the shared prefix and decode with modified scores, one captured graph
replayed step after step with only the lengths, rows and queries changing.

The reference keeps every sequence's K/V in a plain list on the host and never
looks at a block table."""

import numpy as np
import pytest
import torch

from oracle import modified
from paged_kv_cache_292_gb300 import binding

from paritylib import assert_rounded, captured

pytestmark = pytest.mark.gpu

H, HK, D, BS, PREFIX, ROOM = 8, 2, 64, 16, 8, 96
MODS = dict(softcap=20.0, window=40)
# What happens to each of six sequences: n > 0 tokens, -1 leaves.
SCRIPT = [
    [5, 1, 0, 17, 40, 3],
    [1, 1, 1, 1, 1, 1],
    [-1, 1, 1, 1, -1, 2],
    [7, 1, -1, 1, 33, 1],
    [1, -1, 20, -1, 1, -1],
    [0, 12, 1, 9, 1, 0],
]
# Weights: the prefix's enter their product as bf16; scores, cap and exponentials add less than 2^-13.
WEIGHT_ERROR = 2.0**-8 + 2.0**-13


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("graph", [True, False])
def test_steps(graph):
    rng = np.random.default_rng(11)
    S, NB, MB = len(SCRIPT[0]), 60, PREFIX + 12
    order = rng.permutation(NB).astype(np.int32)
    prefix_rows = (_bf16(rng, PREFIX * BS, HK, D), _bf16(rng, PREFIX * BS, HK, D))
    pools = [torch.full((NB, BS, HK, D), float("nan"), dtype=torch.bfloat16) for _ in range(2)]
    for pool, rows in zip(pools, prefix_rows):
        pool[torch.from_numpy(order[:PREFIX]).long()] = rows.view(PREFIX, BS, HK, D)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    k, v = (x.cuda() for x in pools)
    free = np.full(NB, -1, dtype=np.int32)
    free[: NB - PREFIX] = order[PREFIX:]
    prefix, tables, free_d, count = i32(order[:PREFIX]), i32(np.full((S, MB), -1)), i32(free), i32([NB - PREFIX])
    lens, lens_out, count_out, starts, new = i32([0] * S), i32([0] * S), i32([0]), i32([0] * (S + 1)), i32([0] * S)
    slots = torch.empty(ROOM, dtype=torch.int64, device="cuda")
    k_new, v_new = (torch.zeros(ROOM, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(S, H, D, dtype=torch.bfloat16, device="cuda")
    outs = [torch.full_like(q, float("nan")) for _ in range(2)]
    err = i32([0])
    scale = D**-0.5
    ws = torch.empty(max(binding.pa_decode_prefix_workspace_size(S, 1, H, HK, D),
                         binding.pa_decode_mod_workspace_size(S, 1, H, HK, D, binding.PA_BF16)),
                     dtype=torch.uint8, device="cuda")

    def step():
        binding.tables_step(tables, lens, new, free_d, count, BS, slots, prefix_table=prefix, context_lens_out=lens_out,
                            free_count_out=count_out, seq_starts=starts, error_flag=err)
        binding.write_cache(k_new, v_new, slots, k, v, error_flag=err)
        binding.decode_prefix(q, k, v, prefix, tables, lens_out, scale, out=outs[0], workspace=ws, error_flag=err,
                              check_block_ids=True)
        binding.decode_mod(q, k, v, tables, lens_out, scale, out=outs[1], workspace=ws, error_flag=err,
                           check_block_ids=True, **MODS)
        lens.copy_(lens_out)
        count.copy_(count_out)

    run = captured(step).replay if graph else step
    kept = [None] * S  # (K, V) of each live sequence, prefix included
    for script in SCRIPT:
        rows = (_bf16(rng, ROOM, HK, D), _bf16(rng, ROOM, HK, D))
        queries = _bf16(rng, S, H, D)
        at = 0
        for s, n in enumerate(script):
            if n == -1:
                kept[s] = None
            elif n > 0:
                old = kept[s] or prefix_rows
                kept[s] = tuple(torch.cat([o, r[at : at + n]]) for o, r in zip(old, rows))
                at += n
        for dst, src in ((k_new, rows[0]), (v_new, rows[1]), (q, queries)):
            dst.copy_(src)
        new.copy_(torch.tensor(script, dtype=torch.int32))
        run()
        torch.cuda.synchronize()
        assert int(err) == 0
        ctx = np.array([0 if x is None else len(x[0]) for x in kept])
        assert np.array_equal(lens.cpu().numpy(), ctx)
        live = sum(-(-int(c) // BS) - PREFIX for c in ctx if c)
        assert int(count) == NB - PREFIX - live
        # One block per sequence, as long as the longest of them.
        pool = np.zeros((2, S, ctx.max(), HK, D))
        for s, x in enumerate(kept):
            if x is not None:
                for i in range(2):
                    pool[i, s, : ctx[s]] = x[i].double().numpy()
        q64 = queries.double().numpy()[:, None]
        for out, mods in zip(outs, ({}, MODS)):
            want, spread = modified.decode_mod(q64, pool[0], pool[1], np.arange(S)[:, None], ctx, scale, int(ctx.max()),
                                               **mods)
            assert_rounded(out[:, None], want, spread, WEIGHT_ERROR, f"step {script}")
            assert all(torch.all(out[s] == 0) for s in range(S) if ctx[s] == 0)
