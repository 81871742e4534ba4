"""Bounded waits of chunk attention: a withheld copy ends the call with PA_DEVERR_TIMEOUT instead of a hang, and the
next call on the same scratch is right."""

import time

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

from chunklib import Chunks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


@pytest.mark.parametrize("pool", ["bf16", "int8"])
@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("new, old", [([600, 300], [3000, 5000]), ([1, 2, 16], [9000, 300, 20000])])
@pytest.mark.parametrize("tile", [0, 1, 2, 4])
def test_withheld_copy(pool, bs, new, old, tile):
    """Items with two row tiles and with one; the first, the second and a later tile of every CTA.  (The second batch has
    2 KV heads x 231 tiles for 152 CTAs: none takes a fifth, so that call ends as any other.)"""
    b = Chunks(new, old, pool, 8, 2, 128, bs)
    args = b.gpu()
    ws = torch.full((binding.pa_prefill_workspace_size(b.D),), 255, dtype=torch.uint8, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = b.call(args, workspace=ws, error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0
    binding.pa_test_stall_copy(tile, 1000)
    t0 = time.perf_counter()
    b.call(args, workspace=ws, error_flag=flag)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    if tile == 4 and len(new) == 3:
        assert int(flag) == 0
    else:
        assert int(flag) & binding.PA_DEVERR_TIMEOUT
    assert took < 0.5, took  # a few 1 ms limits, not the default 2 s
    flag.zero_()
    out = b.call(args, workspace=ws, error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0
    rows = slice(int(b.starts[0]), int(b.starts[-1]))
    assert torch.equal(out[rows], ref[rows])


@pytest.mark.parametrize("Q", [1, 3])
def test_withheld_copy_of_decode_int8(Q):
    b = Chunks([Q] * 5, [700, 40, 3000, 9, 100], "int8", 8, 2, 128, gap=0)
    q, k, v, ks, vs, tables, lens, _, scale = b.gpu()
    q = q.view(5, Q, 8, 128)
    ws = torch.zeros(binding.pa_decode_int8_workspace_size(5, Q, 8, 2, 128), dtype=torch.uint8, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        return binding.decode_int8(q, k, v, ks, vs, tables, lens, scale, workspace=ws, error_flag=flag)

    ref = call()
    torch.cuda.synchronize()
    assert int(flag) == 0
    for tile in (0, 60, 200):
        binding.pa_test_stall_copy(tile, 1000)
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        assert int(flag) & binding.PA_DEVERR_TIMEOUT and time.perf_counter() - t0 < 0.5
        flag.zero_()
        ws.zero_()
        assert torch.equal(call(), ref)
        torch.cuda.synchronize()
        assert int(flag) == 0
