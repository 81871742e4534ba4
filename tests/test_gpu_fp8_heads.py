"""FP8 pools of 64 dims and every even number of KV heads, which a CTA takes in groups of an even number."""

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle import modified
from paged_kv_cache_292_gb300 import binding

from paritylib import assert_rounded

pytestmark = pytest.mark.gpu

# Weights enter the second product as f16 (half a step); scores and exponentials add less than 2^-13.
WEIGHT_ERROR = 2.0**-11 + 2.0**-13


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


@pytest.mark.parametrize("Hk", [2, 6, 10, 14, 18])
@pytest.mark.parametrize("G, Q", [(1, 1), (4, 1), (3, 3), (5, 4), (8, 4)])
def test_even_numbers_of_kv_heads(Hk, G, Q):
    S, D, bs, nblk = 3, 64, 16, 6
    rng = np.random.default_rng([Hk, G, Q])
    NB = S * nblk
    k, v = (ofp8.quantize(rng.standard_normal((NB, bs, Hk, D)), 0.25) for _ in range(2))
    table = rng.permutation(NB).astype(np.int32).reshape(S, nblk)
    lens = np.array([nblk * bs, 37, Q], dtype=np.int32)
    q = torch.from_numpy(rng.standard_normal((S, Q, G * Hk, D), dtype=np.float32)).to(torch.bfloat16)
    cuda = [torch.from_numpy(x).cuda() for x in (k, v, table, lens)]
    out = binding.decode_fp8_multi(q.cuda(), *cuda, D**-0.5, 0.25, 0.25)
    torch.cuda.synchronize()
    values = [ofp8.e4m3_decode(x) * 0.25 for x in (k, v)]
    want, spread = modified.decode_mod(q.double().numpy(), *values, table, lens, D**-0.5, bs)
    assert_rounded(out, want, spread, WEIGHT_ERROR, f"{Hk} KV heads")
