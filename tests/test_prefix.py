"""pa_decode_prefix on the CPU: its refusals."""

import os
import subprocess

import pytest
import torch

from paged_kv_cache_292_gb300 import binding
from paged_kv_cache_292_gb300 import build as pa_build

INVALID, UNSUPPORTED = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return binding.load()


def _args(**kw):
    a = dict(out=16, query=16, k_cache=16, v_cache=16, prefix_table=16, block_tables=16, context_lens=16, num_seqs=1,
             num_queries=1, num_heads=8, num_kv_heads=8, head_size=128, block_size=16, num_prefix_blocks=2,
             max_blocks_per_seq=4, scale=0.1, stream=0, dtype=binding.PA_BF16, num_physical_blocks=0, workspace=None,
             workspace_bytes=0, error_flag=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw, code", [
    *[({name: None}, INVALID) for name in ("out", "query", "k_cache", "v_cache", "prefix_table", "block_tables",
                                           "context_lens")],
    (dict(num_prefix_blocks=-1), INVALID),
    (dict(num_prefix_blocks=5), INVALID),  # longer than a row
    (dict(prefix_table=18), INVALID),
    (dict(dtype=binding.PA_F32), UNSUPPORTED),
    (dict(dtype=binding.PA_FP8_E4M3), UNSUPPORTED),
    (dict(block_size=12), UNSUPPORTED),
    (dict(block_size=1), UNSUPPORTED),
    (dict(block_size=0), INVALID),
    (dict(block_size=8192), UNSUPPORTED),
    (dict(num_queries=0), INVALID),
    (dict(num_queries=33), UNSUPPORTED),
    (dict(num_heads=72, num_kv_heads=8), UNSUPPORTED),  # group 9
    (dict(num_heads=32, num_kv_heads=8, num_queries=9), UNSUPPORTED),  # 36 columns
    (dict(num_heads=12), INVALID),
    (dict(num_seqs=0), INVALID),
    (dict(head_size=96), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID),
    (dict(k_cache=24), INVALID),
])
def test_rejects_bad_arguments_on_host(lib, kw, code):
    assert lib.pa_decode_prefix(*_args(**kw)) == code
    assert lib.pa_last_error().decode()


def test_workspace_size_of_invalid_sizes_is_zero(lib):
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 9, 8, 128), (1, 1, 8, 0, 128), (1, 1, 8, 8, 0)):
        assert binding.pa_decode_prefix_workspace_size(*bad) == 0


def test_python_layer_wants_cuda_tensors():
    q = torch.zeros(1, 8, 64, dtype=torch.bfloat16)
    pool = torch.zeros(2, 16, 8, 64, dtype=torch.bfloat16)
    one = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.decode_prefix(q, pool, pool, one, one.view(1, 1), one, 0.125)


def test_work_decomposition_host_check(tmp_path):
    """Every tile has one CTA, partial slots never collide, the join finds them (plain C++ build of the header)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "prefix_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I" + os.path.join(root, "paged_kv_cache_292_gb300", "csrc"),
                    os.path.join(root, "tests", "host", "prefix_check.cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok")


def _fp8_args(**kw):
    a = dict(zip(("out query k_cache v_cache prefix_table block_tables context_lens num_seqs num_queries num_heads "
                  "num_kv_heads head_size block_size num_prefix_blocks max_blocks_per_seq scale").split(), _args()))
    a.update(k_scale=0.5, v_scale=2.0, stream=0, num_physical_blocks=0, workspace=None, workspace_bytes=0,
             error_flag=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw, code", [
    *[({name: None}, INVALID) for name in ("out", "query", "k_cache", "v_cache", "prefix_table", "block_tables",
                                           "context_lens")],
    *[({name: bad}, INVALID) for name in ("k_scale", "v_scale") for bad in (0.0, -1.0, float("nan"), float("inf"))],
    (dict(num_prefix_blocks=5), INVALID),
    (dict(block_size=12), UNSUPPORTED),
    (dict(num_queries=33), UNSUPPORTED),
    (dict(num_heads=3, num_kv_heads=3, head_size=64), UNSUPPORTED),
    (dict(head_size=96), UNSUPPORTED),
    (dict(k_cache=24), INVALID),
])
def test_fp8_rejects_bad_arguments_on_host(lib, kw, code):
    assert lib.pa_decode_fp8_prefix(*_fp8_args(**kw)) == code
    assert lib.pa_last_error().decode()
