"""Pools of more than 2^32 bytes (bf16: more than 2^31 elements) whose blocks in use lie at both ends: the results of
every decode are those of the same blocks gathered into a small pool."""

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

pytestmark = pytest.mark.gpu

S, Q, Hk, G, D, bs, nblk = 5, 2, 8, 4, 128, 16, 9


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_blocks_behind_32_bits(kind):
    dtype = {"bf16": torch.bfloat16, "fp8": torch.uint8, "f32": torch.float32}[kind]
    block = bs * Hk * D
    NB = (5 << 30) // (block * dtype.itemsize)
    used = S * nblk
    ids = torch.cat([torch.arange(used // 2), NB - used + used // 2 + torch.arange(used - used // 2)])
    assert int(ids.max()) == NB - 1
    gen = torch.Generator().manual_seed(8)
    order = torch.randperm(used, generator=gen)
    large, small = [], []
    for _ in range(2):
        if kind == "fp8":
            values = torch.randint(0, 0x60, (used, bs, Hk, D), generator=gen, dtype=torch.uint8).cuda()
        else:
            values = torch.randn(used, bs, Hk, D, generator=gen).to(dtype).cuda()
        pool = torch.empty(NB, bs, Hk, D, dtype=dtype, device="cuda")
        pool[ids.cuda()] = values
        large.append(pool)
        small.append(values)
    small_table = order.to(torch.int32).view(S, nblk)
    small_table[:, :2] = small_table[0, :2].clone()
    large_table = ids[small_table.long()].to(torch.int32).cuda()
    small_table = small_table.cuda()
    lens = torch.tensor([nblk * bs, 3 * bs, nblk * bs - 5, 2 * bs + 2, 100], dtype=torch.int32).cuda()
    queries = 1 if kind == "f32" else Q
    q = torch.randn(S, queries, G * Hk, D, generator=gen).to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()

    def calls(pools, table):
        args = (q, *pools, table, lens, D**-0.5)
        if kind == "f32":
            return [binding.decode_mod(*args, softcap=20.0, window=60), binding.decode(q[:, 0].contiguous(), *args[1:])]
        prefix = table[0, :2].contiguous()
        if kind == "fp8":
            return [binding.decode_fp8_multi(*args, 0.5, 2.0), binding.decode_fp8_mod(*args, 0.5, 2.0, window=60),
                    binding.decode_fp8_prefix(q, *pools, prefix, table, lens, D**-0.5, 0.5, 2.0)]
        return [binding.decode_multi(*args), binding.decode_mod(*args, window=60),
                binding.decode_prefix(q, *pools, prefix, table, lens, D**-0.5)]

    for a, b in zip(calls(large, large_table), calls(small, small_table)):
        torch.cuda.synchronize()
        assert torch.isfinite(a.float()).all()
        assert torch.equal(a, b)
