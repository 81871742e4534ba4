"""Bounded waits of the shared-prefix kernel and of the walk with modified scores:
a withheld copy ends the call with PA_DEVERR_TIMEOUT instead of a hang, and the
next call on the same scratch is right."""

import time

import numpy as np
import pytest
import torch

from paged_kv_cache_292_gb300 import binding, workloads

from paritylib import to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _prefix_call(heads, D, S):
    """A batch of S sequences of a few tokens behind 512 shared ones; (tiles of the prefix kernel, call, scratch)."""
    kv_heads, bs, blocks = 2, 16, 32
    gen = torch.Generator().manual_seed(5)
    pools = [torch.randn(blocks + S, bs, kv_heads, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    prefix = torch.arange(blocks, dtype=torch.int32)
    tables = torch.cat([prefix.expand(S, -1), (blocks + torch.arange(S, dtype=torch.int32))[:, None]], 1).contiguous()
    q = torch.randn(S, heads, D, generator=gen).to(torch.bfloat16).cuda()
    lens = torch.full((S,), blocks * bs + 3, dtype=torch.int32).cuda()
    ws = torch.full((binding.pa_decode_prefix_workspace_size(S, 1, heads, kv_heads, D),), 255, dtype=torch.uint8,
                    device="cuda")
    prefix, tables = prefix.cuda(), tables.cuda()
    items = kv_heads * -(-S * (heads // kv_heads) // 256)

    def call(flag):
        return binding.decode_prefix(q, *pools, prefix, tables, lens, D**-0.5, workspace=ws, error_flag=flag)

    return items * 4, call


def _mod_call(dtype, Q):
    sp = workloads.spec("llama3_8b", num_seqs=12, ctx_lo=1, ctx_hi=700, max_context=704, pool_blocks=600, dtype=dtype)
    w = workloads.make_workload(sp, prewritten=True)
    g = to_device(w)
    S, H, D = w.q.shape
    q = g["q"] if Q == 1 else torch.randn(S, Q, H, D, generator=torch.Generator().manual_seed(3)).to(w.q.dtype).cuda()
    kv = binding.PA_F32 if dtype == "f32" else binding.PA_BF16
    ws = torch.full((binding.pa_decode_mod_workspace_size(S, Q, H, 8, D, kv),), 255, dtype=torch.uint8, device="cuda")

    def call(flag):
        return binding.decode_mod(q, g["k_cache"], g["v_cache"], g["block_tables"], g["context_lens"], w.scale,
                                  softcap=20.0, workspace=ws, error_flag=flag)

    return int(sum(-(-int(c) // 16) for c in w.context_lens.tolist())), call


CALLS = {
    "prefix, one row tile": lambda: _prefix_call(8, 128, 10),
    "prefix, two row tiles": lambda: _prefix_call(8, 64, 60),
    "prefix, three row tiles": lambda: _prefix_call(8, 128, 90),
    "mod": lambda: _mod_call("bf16", 1),
    "mod, 16 columns": lambda: _mod_call("bf16", 4),
    "mod, fp32": lambda: _mod_call("f32", 1),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_withheld_copy_times_out_and_the_next_call_is_clean(name, where):
    tiles, call = CALLS[name]()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = call(flag)
    torch.cuda.synchronize()
    assert int(flag) == 0 and np.isfinite(ref.float().cpu().numpy()).all()
    binding.pa_test_stall_copy(min(int(where * tiles), tiles - 1), 1000)
    t0 = time.perf_counter()
    call(flag)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert int(flag) == binding.PA_DEVERR_TIMEOUT
    assert took < 0.5, took  # a few 1 ms limits, not the default 2 s
    flag.zero_()
    out = call(flag)
    torch.cuda.synchronize()
    assert int(flag) == 0
    assert torch.equal(out, ref)
