"""Bounded waits of the walk behind a shared prefix: a withheld copy of one of its tiles ends the call with
PA_DEVERR_TIMEOUT instead of a hang, beside the prefix kernel or alone, and the next call on the same scratch is right."""

import time

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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D, Q", [(128, 2), (64, 2), (128, 4), (64, 4)])  # 8 and 16 columns per KV head
@pytest.mark.parametrize("blocks", [0, 32])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_withheld_copy_of_the_walk(fp8, D, Q, blocks, where):
    Hk, G, bs, S, own = 2, 4, 16, 40, 3
    gen = torch.Generator().manual_seed(6)
    NB = blocks + S * own
    shape = (NB, bs, Hk, D)
    if fp8:
        pools = [torch.randint(0, 0x60, shape, generator=gen, dtype=torch.uint8).cuda() for _ in range(2)]
    else:
        pools = [torch.randn(shape, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    prefix = torch.arange(blocks, dtype=torch.int32)
    rows = blocks + torch.arange(S * own, dtype=torch.int32).view(S, own)
    tables = torch.cat([prefix.expand(S, -1), rows], 1).contiguous().cuda()
    lens = torch.full((S,), (blocks + own) * bs, dtype=torch.int32).cuda()
    q = torch.randn(S, Q, G * Hk, D, generator=gen).to(torch.bfloat16).cuda()
    ws = torch.full((binding.pa_decode_prefix_workspace_size(S, Q, G * Hk, Hk, D),), 255, dtype=torch.uint8,
                    device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    fn, scales = (binding.decode_fp8_prefix, (0.5, 2.0)) if fp8 else (binding.decode_prefix, ())

    def call():
        return fn(q, *pools, prefix.cuda(), tables, lens, D**-0.5, *scales, workspace=ws, error_flag=flag)

    ref = call()
    torch.cuda.synchronize()
    assert int(flag) == 0 and torch.isfinite(ref.float()).all()
    prefix_tiles = -(-blocks * bs // 128) * Hk * -(-S * Q * G // 256)
    walk_tiles = S * own
    binding.pa_test_stall_copy(prefix_tiles + min(int(where * walk_tiles), walk_tiles - 1), 1000)
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert int(flag) == binding.PA_DEVERR_TIMEOUT
    assert took < 0.5, took  # a few 1 ms limits, not the default 2 s
    flag.zero_()
    out = call()
    torch.cuda.synchronize()
    assert int(flag) == 0
    assert torch.equal(out, ref)
