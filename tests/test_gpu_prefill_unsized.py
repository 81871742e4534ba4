"""pa_prefill without the pools' size (num_physical_blocks = 0): the rows that the driver knows of bound the tensor
maps and the block ids, and results are those of the call that gives the size."""

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

from chunklib import Chunks

pytestmark = pytest.mark.gpu

BYTES = 24 << 20  # whole 2 MiB pages


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _inside(pool, behind):
    """The pool `behind` bytes before the end of an allocation of its own (NaN around it)."""
    size = pool.numel() * pool.element_size()
    arena = torch.full((BYTES,), 255, dtype=torch.uint8, device="cuda")
    view = arena[BYTES - behind - size : BYTES - behind].view(pool.dtype).view(pool.shape)
    view.copy_(pool)
    return view


def _call(b, q, k, v, tables, blocks, flag):
    S, MB = tables.shape
    out = torch.full_like(q, 77.0)
    lens, starts = b.gpu()[-3:-1]
    binding.pa_prefill(out, q, k, v, tables, lens, starts, b.T, S, b.heads, k.shape[2], b.D, b.bs, MB, b.scale, None, None,
                       blocks, None, 0, flag)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("bs, D, kv_heads", [(16, 128, 2), (5, 64, 3), (8, 64, 1), (40, 128, 1)])
@pytest.mark.parametrize("behind_k, behind_v", [(0, 0), (16 * 37, 0), (0, 16 * 1001), (5 << 20, 6 << 20)])
def test_rows_from_the_driver(pool, bs, D, kv_heads, behind_k, behind_v):
    b = Chunks([70, 1, 0, 300], [100, 400, 30, 0], pool, 4 * kv_heads, kv_heads, D, bs)
    args = b.gpu()
    q, tables = args[0], args[3]
    k, v = _inside(args[1], behind_k), _inside(args[2], behind_v)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = _call(b, q, k, v, tables, k.shape[0], flag)
    rows = b.compare(want, "with the size")
    got = _call(b, q, k, v, tables, 0, flag)
    assert int(flag) == 0
    assert torch.equal(got, want)
    assert bool((got[torch.from_numpy(~rows).cuda()] == 77.0).all())


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("bad", [2**31 - 1, 2**30, -1, -(2**31)])
def test_ids_beyond_the_memory_are_reported(pool, bs, bad):
    """No id of these is a row of any allocation; the other sequence is right."""
    b = Chunks([40, 60], [100, 30], pool, 8, 2, 128, bs)
    args = b.gpu()
    q, k, v, tables = args[:4]
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = _call(b, q, k, v, tables, 0, flag)
    assert int(flag) == 0
    tables = tables.clone()
    tables[0, 1] = bad
    got = _call(b, q, k, v, tables, 0, flag)
    assert int(flag) == binding.PA_DEVERR_BLOCK_ID
    rows = slice(int(b.starts[1]), int(b.starts[2]))
    assert torch.equal(got[rows], want[rows])
