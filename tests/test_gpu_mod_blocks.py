"""Modified scores over blocks of every small size with many columns per KV head: staged rows of blocks that are no
multiple of 4 take more shared memory, and plans that do not fit give way to others instead of a refusal."""

import numpy as np
import pytest
import torch

from oracle import modified
from paged_kv_cache_292_gb300 import binding

from paritylib import assert_rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


@pytest.mark.parametrize("bs", [1, 2, 3, 6, 10, 12])
@pytest.mark.parametrize("Hk, G, Q", [(4, 6, 4), (8, 8, 3), (7, 5, 3), (5, 4, 8)])  # 24, 24, 15 and 32 columns
@pytest.mark.parametrize("fp8", [False, True])
def test_small_blocks_and_many_columns(bs, Hk, G, Q, fp8):
    S, D, c = 2, 128, 75
    nblk = -(-c // bs)
    NB = S * nblk
    rng = np.random.default_rng([bs, Hk, G, Q])
    table = rng.permutation(NB).astype(np.int32).reshape(S, nblk)
    lens = np.array([c, 33], dtype=np.int32)
    q = torch.from_numpy(rng.standard_normal((S, Q, G * Hk, D), dtype=np.float32)).to(torch.bfloat16)
    mods = dict(softcap=20.0, window=41)
    if fp8:
        # Codes of finite values up to 1.875; the weights enter the second product as f16 (half a step).
        pools = [rng.integers(0, 0x40, (NB, bs, Hk, D), dtype=np.uint8) for _ in range(2)]
        from oracle import fp8 as ofp8

        values, error = [ofp8.e4m3_decode(x) for x in pools], 2.0**-11 + 2.0**-13
        run = lambda *a: binding.decode_fp8_mod(*a[:5], D**-0.5, 1.0, 1.0, **mods)  # noqa: E731
        gpu = [torch.from_numpy(x).cuda() for x in pools]
    else:
        pools = [torch.from_numpy(rng.standard_normal((NB, bs, Hk, D), dtype=np.float32)).to(torch.bfloat16)
                 for _ in range(2)]
        values, error = [x.double().numpy() for x in pools], 2.0**-13
        run = lambda *a: binding.decode_mod(*a[:5], D**-0.5, **mods)  # noqa: E731
        gpu = [x.cuda() for x in pools]
    out = run(q.cuda(), *gpu, torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda())
    torch.cuda.synchronize()
    want, spread = modified.decode_mod(q.double().numpy(), *values, table, lens, D**-0.5, bs, **mods)
    assert_rounded(out, want, spread, error, f"bs={bs}")
