"""FP8 pools: many tokens far below one dominant token keep their share of the output.

One key of the context scores about 17.5 above all others, which score 0, and its value is 0; theirs is 1.  The
others' weights are 2^-25.25 of the largest, and 128 k of them make up 0.3% of the sum: the whole output.  Each weight
is off by at most 2^-11 of itself, scores and exponentials add less than 2^-13, and the output is rounded once."""

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from paged_kv_cache_292_gb300 import binding

from paritylib import assert_rounded

pytestmark = pytest.mark.gpu

WEIGHT_ERROR = 2.0**-11 + 2.0**-13
D, Hk, bs = 64, 2, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


@pytest.mark.parametrize("tokens", [4096, 1 << 17])
@pytest.mark.parametrize("G, Q", [(4, 1), (4, 2), (8, 2)])  # 4, 8 and 16 columns per KV head
@pytest.mark.parametrize("sink", [0, 77])
def test_weak_tokens_count(tokens, G, Q, sink):
    S, own = 2, 16
    P = tokens // bs
    NB = P + S
    one = int(ofp8.quantize(np.ones(1), 1.0)[0])
    k = torch.zeros(NB, bs, Hk, D, dtype=torch.uint8)
    v = torch.full_like(k, one)
    k[sink // bs, sink % bs] = one
    v[sink // bs, sink % bs] = 0
    # q . k of the dominant token: 64 * 0.2734375 = 17.5
    q = torch.full((S, Q, G * Hk, D), 0.2734375, dtype=torch.bfloat16)
    prefix = torch.arange(P, dtype=torch.int32)
    table = torch.cat([prefix.expand(S, -1), P + torch.arange(S, dtype=torch.int32)[:, None]], 1).contiguous()
    lens = torch.full((S,), tokens + own, dtype=torch.int32)
    gpu = [x.cuda() for x in (q, k, v, prefix, table, lens)]
    q, k, v, prefix, table, lens = gpu
    # Query i sees the tokens up to its own: tokens + own - Q + i + 1 of them, one dominant.
    weak = tokens + own - Q + np.arange(Q, dtype=np.float64)
    share = weak * np.exp(-17.5) / (1 + weak * np.exp(-17.5))
    want = np.broadcast_to(share[None, :, None, None], (S, Q, G * Hk, D))
    for name, out in (
        ("plain", binding.decode_fp8_multi(q, k, v, table, lens, 1.0, 1.0, 1.0)),
        ("modified", binding.decode_fp8_mod(q, k, v, table, lens, 1.0, 1.0, 1.0)),
        ("prefix", binding.decode_fp8_prefix(q, k, v, prefix, table, lens, 1.0, 1.0, 1.0)),
    ):
        torch.cuda.synchronize()
        assert_rounded(out, want, want, WEIGHT_ERROR, f"{name} {tokens}")
