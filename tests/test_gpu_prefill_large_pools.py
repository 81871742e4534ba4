"""Chunk attention and the int8 cache over pools of more than 2^32 bytes whose blocks in use lie at both ends: the results are
those of the same blocks gathered into a small pool."""

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

pytestmark = pytest.mark.gpu

S, Hk, G, D, nblk = 4, 8, 3, 128, 9


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


@pytest.mark.parametrize("bs", [16, 12])
@pytest.mark.parametrize("kind", ["bf16", "f32", "int8"])
def test_blocks_behind_32_bits(kind, bs):
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}[kind]
    NB = (5 << 30) // (bs * Hk * D * dtype.itemsize)
    used = S * nblk
    ids = torch.cat([torch.arange(used // 2), NB - used + used // 2 + torch.arange(used - used // 2)])
    gen = torch.Generator().manual_seed(8)
    order = torch.randperm(used, generator=gen).to(torch.int32).view(S, nblk)
    small_table, large_table = order.cuda(), ids[order.long()].to(torch.int32).cuda()
    new = torch.tensor([50, 1, 30, 0])
    lens = torch.tensor([nblk * bs, 3 * bs - 1, 60, 40], dtype=torch.int32).cuda()
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32).cuda()
    T = int(starts[-1])
    q = torch.randn(T, G * Hk, D, generator=gen).to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()
    results = []
    for blocks, table in ((NB, large_table), (used, small_table)):
        if kind == "int8":
            pools = [torch.zeros(blocks, bs, Hk, D, dtype=torch.int8, device="cuda") for _ in range(2)]
            pools += [torch.zeros(blocks, Hk, bs, device="cuda") for _ in range(2)]
            rows = [torch.randn(used * bs, Hk, D, generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
            at = ids.cuda() if blocks == NB else torch.arange(used).cuda()
            slots = (at[:, None] * bs + torch.arange(bs).cuda()).flatten()
            binding.write_cache_int8(*rows, slots, *pools)
            out = binding.prefill_int8(q, *pools, table, lens, starts, D**-0.5)
            back = [torch.zeros(T, Hk, D, device="cuda") for _ in range(2)]
            binding.read_cache_int8(*pools, table, starts, *back)
            step = binding.decode_int8(q[:S].contiguous(), *pools, table, lens, D**-0.5)
            results.append([out, step, *back])
        else:
            pools = []
            for i in range(2):
                pool = torch.empty(blocks, bs, Hk, D, dtype=dtype, device="cuda")
                values = torch.randn(used, bs, Hk, D, generator=torch.Generator().manual_seed(i)).to(dtype).cuda()
                pool[ids.cuda() if blocks == NB else torch.arange(used).cuda()] = values
                pools.append(pool)
            results.append([binding.prefill(q, *pools, table, lens, starts, D**-0.5)])
        torch.cuda.synchronize()
        del pools
    for a, b in zip(*results):
        assert torch.isfinite(a.float()).all()
        assert torch.equal(a, b)
