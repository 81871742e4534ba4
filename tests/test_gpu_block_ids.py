"""The Python layer gives the library the pools' size: block ids outside the pools are skipped and reported whether
or not the caller asks for the check, and the other sequences' rows are right."""

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


@pytest.mark.parametrize("bad", [-1, 40, 2**31 - 1])
@pytest.mark.parametrize("Q", [1, 3])
@pytest.mark.parametrize("fp8", [False, True])
def test_ids_outside_the_pools(bad, Q, fp8):
    S, Hk, G, D, bs, n = 4, 2, 4, 64, 16, 10
    NB = S * n
    gen = torch.Generator().manual_seed(1)
    if fp8:
        pools = [torch.randint(0, 0x60, (NB, bs, Hk, D), generator=gen, dtype=torch.uint8).cuda() for _ in range(2)]
    else:
        pools = [torch.randn(NB, bs, Hk, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    table = torch.randperm(NB, generator=gen).to(torch.int32).view(S, n).cuda()
    lens = torch.full((S,), n * bs - 3, dtype=torch.int32).cuda()
    q = torch.randn(S, Q, G * Hk, D, generator=gen).to(torch.bfloat16).cuda()
    scales = (0.5, 2.0) if fp8 else ()
    for fn in ((binding.decode_fp8_multi, binding.decode_fp8_mod) if fp8 else
               (binding.decode_multi, binding.decode_mod)):
        good = fn(q, *pools, table, lens, D**-0.5, *scales)
        broken = table.clone()
        broken[2, 4] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = fn(q, *pools, broken, lens, D**-0.5, *scales, error_flag=err)
        torch.cuda.synchronize()
        assert int(err) == binding.PA_DEVERR_BLOCK_ID
        rest = [0, 1, 3]
        assert torch.equal(out[rest], good[rest])
