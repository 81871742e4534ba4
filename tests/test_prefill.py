"""Chunk attention and the int8 cache on the CPU: refusals, the work decomposition, the oracle's pins."""

import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import chunks
from paged_kv_cache_292_gb300 import binding
from paged_kv_cache_292_gb300 import build as pa_build

INVALID, UNSUPPORTED = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return binding.load()


def _prefill(**kw):
    a = dict(out=16, query=16, k_cache=16, v_cache=16, block_tables=16, context_lens=16, seq_starts=16, num_tokens=4,
             num_seqs=1, num_heads=8, num_kv_heads=8, head_size=128, block_size=16, max_blocks_per_seq=4, scale=0.1,
             stream=0, dtype=binding.PA_BF16, num_physical_blocks=8, workspace=None, workspace_bytes=0, error_flag=None)
    a.update(kw)
    return list(a.values())


def _prefill_int8(**kw):
    a = dict(out=16, query=16, k_cache=16, v_cache=16, k_scales=16, v_scales=16, block_tables=16, context_lens=16,
             seq_starts=16, num_tokens=4, num_seqs=1, num_heads=8, num_kv_heads=8, head_size=128, block_size=16,
             max_blocks_per_seq=4, scale=0.1, stream=0, num_physical_blocks=8, workspace=None, workspace_bytes=0,
             error_flag=None)
    a.update(kw)
    return list(a.values())


def _decode_int8(**kw):
    a = dict(out=16, query=16, k_cache=16, v_cache=16, k_scales=16, v_scales=16, block_tables=16, context_lens=16,
             num_seqs=1, num_queries=1, num_heads=8, num_kv_heads=8, head_size=128, block_size=16, max_blocks_per_seq=4,
             scale=0.1, stream=0, num_physical_blocks=8, workspace=None, workspace_bytes=0,
             num_ranges=0, error_flag=None)
    a.update(kw)
    return list(a.values())


SHARED = [
    *[({name: None}, INVALID) for name in ("out", "query", "k_cache", "v_cache", "block_tables", "context_lens")],
    *[({name: 24}, INVALID) for name in ("out", "query", "k_cache", "v_cache")],
    (dict(context_lens=18), INVALID),
    (dict(num_seqs=0), INVALID),
    (dict(num_heads=12), INVALID),
    (dict(num_heads=72), UNSUPPORTED),  # group 9
    (dict(head_size=96), UNSUPPORTED),
    (dict(head_size=0), INVALID),
    (dict(block_size=0), INVALID),
    (dict(block_size=8192), UNSUPPORTED),
    (dict(max_blocks_per_seq=1 << 27), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(num_physical_blocks=-1), INVALID),
]
RAGGED = [(dict(seq_starts=None), INVALID), (dict(seq_starts=18), INVALID), (dict(num_tokens=-1), INVALID),
          (dict(num_tokens=1 << 30), UNSUPPORTED)]
SCALED = [(dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID), (dict(k_scales=20), INVALID),
          (dict(num_physical_blocks=0), INVALID)]


@pytest.mark.parametrize("kw, code", SHARED + RAGGED + [(dict(dtype=binding.PA_FP8_E4M3), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED)])
def test_prefill_rejects(lib, kw, code):
    assert lib.pa_prefill(*_prefill(**kw)) == code
    assert lib.pa_last_error().decode()


@pytest.mark.parametrize("kw, code", SHARED + RAGGED + SCALED)
def test_prefill_int8_rejects(lib, kw, code):
    assert lib.pa_prefill_int8(*_prefill_int8(**kw)) == code
    assert lib.pa_last_error().decode()


@pytest.mark.parametrize("kw, code", SHARED + SCALED + [(dict(num_queries=0), INVALID), (dict(num_queries=1 << 29), UNSUPPORTED),
                                                         (dict(num_ranges=-1), INVALID), (dict(num_ranges=5000), UNSUPPORTED)])
def test_decode_int8_rejects(lib, kw, code):
    assert lib.pa_decode_int8(*_decode_int8(**kw)) == code
    assert lib.pa_last_error().decode()


def _write(**kw):
    a = dict(k_new=16, v_new=16, slot_mapping=16, k_cache=16, v_cache=16, k_scales=16, v_scales=16, num_tokens=1,
             num_kv_heads=2, head_size=128, block_size=16, num_physical_blocks=4, stream=0, src_dtype=binding.PA_BF16,
             error_flag=None)
    a.update(kw)
    return list(a.values())


def _read(**kw):
    a = dict(k_out=16, v_out=16, k_cache=16, v_cache=16, k_scales=16, v_scales=16, block_tables=16, first_tokens=None,
             seq_starts=16, num_tokens=1, num_seqs=1, num_kv_heads=2, head_size=128, block_size=16, max_blocks_per_seq=4,
             num_physical_blocks=4, stream=0, dst_dtype=binding.PA_BF16, error_flag=None)
    a.update(kw)
    return list(a.values())


BOTH = [
    *[({name: None}, INVALID) for name in ("k_cache", "v_cache", "k_scales", "v_scales")],
    (dict(k_cache=24), INVALID),
    (dict(v_scales=18), INVALID),
    (dict(num_tokens=-1), INVALID),
    (dict(num_kv_heads=0), INVALID),
    (dict(num_kv_heads=1 << 20), UNSUPPORTED),
    (dict(head_size=80), UNSUPPORTED),
    (dict(block_size=0), INVALID),
    (dict(block_size=5000), UNSUPPORTED),
    (dict(num_physical_blocks=0), INVALID),
]


@pytest.mark.parametrize("kw, code", BOTH + [(dict(k_new=None), INVALID), (dict(v_new=24), INVALID), (dict(slot_mapping=None), INVALID),
                                             (dict(slot_mapping=20), INVALID), (dict(src_dtype=binding.PA_FP8_E4M3), UNSUPPORTED)])
def test_write_rejects(lib, kw, code):
    assert lib.pa_write_cache_int8(*_write(**kw)) == code
    assert lib.pa_last_error().decode()


@pytest.mark.parametrize("kw, code", BOTH + [(dict(k_out=None), INVALID), (dict(v_out=24), INVALID), (dict(block_tables=None), INVALID),
                                             (dict(seq_starts=None), INVALID), (dict(first_tokens=18), INVALID), (dict(num_seqs=0), INVALID),
                                             (dict(max_blocks_per_seq=0), INVALID), (dict(max_blocks_per_seq=1 << 27), INVALID),
                                             (dict(dst_dtype=7), UNSUPPORTED)])
def test_read_rejects(lib, kw, code):
    assert lib.pa_read_cache_int8(*_read(**kw)) == code
    assert lib.pa_last_error().decode()


def test_calls_without_a_token_do_nothing(lib):
    assert lib.pa_prefill(*_prefill(num_tokens=0)) == binding.PA_OK
    assert lib.pa_prefill(*_prefill(num_tokens=0, out=None, query=None)) == binding.PA_OK
    assert lib.pa_prefill(*_prefill(num_tokens=0, k_cache=None)) == INVALID
    assert lib.pa_write_cache_int8(*_write(num_tokens=0, k_new=None, v_new=None, slot_mapping=None)) == binding.PA_OK
    assert lib.pa_read_cache_int8(*_read(num_tokens=0, k_out=None, v_out=None)) == binding.PA_OK


def test_workspace_size_of_an_invalid_head_size_is_zero(lib):
    assert binding.pa_prefill_workspace_size(96) == 0
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 9, 8, 128), (1, 1, 8, 0, 128), (1, 1, 8, 8, 96), (1, 1, 8, 8, 128, -1)):
        assert binding.pa_decode_int8_workspace_size(*bad) == 0


def test_python_layer_wants_cuda_tensors():
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    pool = torch.zeros(2, 16, 8, 64, dtype=torch.bfloat16)
    codes, scales = pool.to(torch.int8), torch.zeros(2, 8, 16)
    one, starts = torch.ones(1, dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.prefill(q, pool, pool, one.view(1, 1), one, starts, 0.125)
    with pytest.raises(ValueError):
        binding.prefill_int8(q, codes, codes, scales, scales, one.view(1, 1), one, starts, 0.125)
    with pytest.raises(ValueError):
        binding.decode_int8(q, codes, codes, scales, scales, one.view(1, 1), one, 0.125)
    with pytest.raises(ValueError):
        binding.write_cache_int8(q, q, torch.zeros(2, dtype=torch.int64), codes, codes, scales, scales)
    with pytest.raises(ValueError):
        binding.read_cache_int8(codes, codes, scales, scales, one.view(1, 1), starts, q, q)


def test_work_decomposition_host_check(tmp_path):
    """Every tile has one range, at most one item is cut at either end of it, the join finds the parts."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "chunk_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I" + os.path.join(root, "paged_kv_cache_292_gb300", "csrc"),
                    os.path.join(root, "tests", "host", "chunk_check.cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok")


# ---- the oracle ------------------------------------------------------------------


def test_oracle_prefill_is_multi_query_decode():
    """Equal chunks are the multi-query decode that has pins of its own; each sequence alone gives the same rows."""
    rng = np.random.default_rng(0)
    S, Q, H, Hk, D, bs = 3, 5, 4, 2, 8, 4
    ctx = np.array([5, 17, 3])
    tables = rng.permutation(15).reshape(3, 5)
    k, v = rng.standard_normal((2, 15, bs, Hk, D))
    q = rng.standard_normal((S, Q, H, D))
    out, spread, reach = chunks.prefill(q.reshape(S * Q, H, D), k, v, tables, ctx, np.arange(S + 1) * Q, 0.4, bs)
    np.testing.assert_allclose(out.reshape(q.shape), oracle.decode_multi(q, k, v, tables, ctx, 0.4, bs), atol=1e-12)
    assert (spread >= np.abs(out) - 1e-12).all() and (reach >= 0).all()
    ragged = chunks.prefill(q.reshape(S * Q, H, D), k, v, tables[1:2], ctx[1:2], [6, 9], 0.4, bs)[0]
    assert np.isnan(ragged[:6]).all() and np.isnan(ragged[9:]).all()
    one = chunks.prefill(q.reshape(S * Q, H, D)[6:9], k, v, tables[1:2], ctx[1:2], [0, 3], 0.4, bs)[0]
    np.testing.assert_allclose(ragged[6:9], one, atol=0)


def test_oracle_quantise_in_rationals():
    """Codes by exact arithmetic on ties, next to them, and on random rows."""
    rng = np.random.default_rng(1)
    rows = [rng.standard_normal(16).astype(np.float32) * np.float32(s) for s in (1e-30, 1e-3, 1, 7e5)]
    rows.append(np.array([127, 2.5, -2.5, 3.5, 0.5, -0.5, np.nextafter(np.float32(2.5), 9, dtype=np.float32), 1], dtype=np.float32))
    for x in rows:
        codes, scale = chunks.quantise(x)
        assert scale == np.float32(np.abs(x).max()) / np.float32(127)
        for c, e in zip(codes, x):
            step = Fraction(float(e)) / Fraction(float(scale))
            assert abs(step - int(c)) <= Fraction(1, 2) and (abs(step - int(c)) < Fraction(1, 2) or int(c) % 2 == 0)
    codes, scale = chunks.quantise(np.array([[0.0, -0.0], [1.0, np.inf], [np.nan, 2.0]], dtype=np.float32))
    assert (codes == 0).all() and scale[0] == 0 and np.isnan(scale[1:]).all()
