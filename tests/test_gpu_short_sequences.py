"""Runs of sequences of one to three tiles (16 tokens) in every order, in kernels
whose ring holds more tiles than the query ring holds sequences: the producer
warps must neither fill a query slot ahead of its turn nor wait for a turn that
has passed."""

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
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


CTX = np.random.default_rng(11).choice([1, 2, 15, 16, 17, 31, 33, 40, 48], 600)
SHAPES = [(8, 2, 64), (32, 8, 64), (32, 8, 128), (64, 8, 128), (8, 1, 128), (10, 10, 128), (5, 5, 128)]


def _batch(heads, kv_heads, head_size, dtype):
    sp = workloads.spec("llama3_8b", num_seqs=len(CTX), num_heads=heads, num_kv_heads=kv_heads, head_size=head_size,
                        max_context=64, pool_blocks=0, dtype=dtype)
    w = workloads.make_workload(sp, prewritten=True, context_lens=CTX)
    return w, to_device(w)


@pytest.mark.parametrize("heads, kv_heads, head_size", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("num_ranges", [0, 1, 7])
def test_decode_and_modified(heads, kv_heads, head_size, dtype, num_ranges):
    w, g = _batch(heads, kv_heads, head_size, dtype)
    args = (g["q"], g["k_cache"], g["v_cache"], g["block_tables"], g["context_lens"], w.scale)
    want, err = oracle_decode(w), torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        for fn, kw in ((binding.decode, {}), (binding.decode_mod, dict(window=4096))):
            out = fn(*args, num_ranges=num_ranges, error_flag=err, **kw)
            torch.cuda.synchronize()
            assert int(err) == 0
            assert_close(out, want, dtype, "short sequences")


@pytest.mark.parametrize("heads, kv_heads, head_size", SHAPES)
def test_behind_a_prefix_of_nothing(heads, kv_heads, head_size):
    w, g = _batch(heads, kv_heads, head_size, "bf16")
    none, err = torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out = binding.decode_prefix(g["q"], g["k_cache"], g["v_cache"], none, g["block_tables"], g["context_lens"],
                                    w.scale, error_flag=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        assert_close(out, oracle_decode(w), "bf16", "short sequences")


@pytest.mark.parametrize("heads, kv_heads, head_size, Q", [(8, 2, 64, 1), (32, 8, 128, 1), (32, 8, 128, 4), (8, 2, 64, 3)])
def test_fp8_and_several_queries_agree(heads, kv_heads, head_size, Q):
    """FP8 and multi-query kernels: the plain step, the walk with modified scores and the walk behind a prefix of
    no tokens do the same sums in other orders."""
    w, g = _batch(heads, kv_heads, head_size, "bf16")
    S = len(CTX)
    q = torch.randn(S, Q, heads, head_size, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    rest = (g["block_tables"], g["context_lens"], w.scale)
    codes = [torch.from_numpy(ofp8.quantize(x.float().numpy(), 0.02)).cuda() for x in (w.k_cache, w.v_cache)]
    none, err = torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        plain = binding.decode_multi(q, g["k_cache"], g["v_cache"], *rest, error_flag=err)
        others = [binding.decode_mod(q, g["k_cache"], g["v_cache"], *rest, error_flag=err),
                  binding.decode_prefix(q, g["k_cache"], g["v_cache"], none, *rest, error_flag=err)]
        plain8 = binding.decode_fp8_multi(q, *codes, *rest, 0.02, 0.02, error_flag=err)
        others8 = [binding.decode_fp8_mod(q, *codes, *rest, 0.02, 0.02, error_flag=err),
                   binding.decode_fp8_prefix(q, *codes, none, *rest, 0.02, 0.02, error_flag=err)]
        torch.cuda.synchronize()
        assert int(err) == 0
        # Two roundings to bf16 (2^-8 together) of values up to the largest |v|, and f16 weights twice.
        for a, b in [(plain, x) for x in others] + [(plain8, x) for x in others8]:
            d = (a.float() - b.float()).abs().max()
            assert torch.isfinite(b.float()).all() and d <= 2.0**-8 * a.float().abs().max() + 2.0**-9 * 8, float(d)
