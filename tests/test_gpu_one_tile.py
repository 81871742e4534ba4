"""Runs of sequences of one tile (16 tokens) each, for group sizes whose queries
leave room for one query slot in shared memory only (bf16, 64 query heads of 128
over 8 KV heads): the decode kernel's two producer warps must not fill the slot
ahead of its turn."""

import numpy as np
import pytest
import torch

from paged_kv_cache_292_gb300 import binding, workloads

from paritylib import assert_close, oracle_decode, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


CTX = np.concatenate([np.arange(160) % 16 + 1, [300, 1, 2, 3], np.full(60, 16)])


def _batch(heads, kv_heads, head_size, dtype):
    sp = workloads.spec("llama3_8b", num_seqs=len(CTX), num_heads=heads, num_kv_heads=kv_heads, head_size=head_size,
                        max_context=304, pool_blocks=0, dtype=dtype)
    w = workloads.make_workload(sp, prewritten=True, poison=True, context_lens=CTX)
    return w, to_device(w)


SHAPES = [(64, 8, 128), (32, 8, 128), (64, 8, 64)]


@pytest.mark.parametrize("heads, kv_heads, head_size", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("num_ranges", [0, 1])
def test_decode(heads, kv_heads, head_size, dtype, num_ranges):
    w, g = _batch(heads, kv_heads, head_size, dtype)
    out = binding.decode(g["q"], g["k_cache"], g["v_cache"], g["block_tables"], g["context_lens"], w.scale,
                         num_ranges=num_ranges)
    torch.cuda.synchronize()
    assert_close(out, oracle_decode(w), dtype, "one-tile sequences")


@pytest.mark.parametrize("heads, kv_heads, head_size", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("num_ranges", [0, 1])
def test_decode_mod(heads, kv_heads, head_size, dtype, num_ranges):
    """The same through the walk with modified scores (a cap far above the scores changes nothing)."""
    w, g = _batch(heads, kv_heads, head_size, dtype)
    out = binding.decode_mod(g["q"], g["k_cache"], g["v_cache"], g["block_tables"], g["context_lens"], w.scale,
                             num_ranges=num_ranges, window=4096)
    torch.cuda.synchronize()
    assert_close(out, oracle_decode(w), dtype, "one-tile sequences")


@pytest.mark.parametrize("heads, kv_heads, head_size", SHAPES)
def test_decode_prefix_of_nothing(heads, kv_heads, head_size):
    """The walk behind a shared prefix, here of no tokens."""
    w, g = _batch(heads, kv_heads, head_size, "bf16")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = binding.decode_prefix(g["q"], g["k_cache"], g["v_cache"], none, g["block_tables"], g["context_lens"], w.scale)
    torch.cuda.synchronize()
    assert_close(out, oracle_decode(w), "bf16", "one-tile sequences")
