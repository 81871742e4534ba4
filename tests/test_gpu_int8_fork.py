"""A forked sequence over the int8 cache: blocks of codes and of scales copied before the child writes into them."""

import numpy as np
import pytest
import torch

from oracle import chunks
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


def _copy(pools, copies):
    """The pools' blocks as 16-bit elements, the scales' as fp32: both are copied bit by bit."""
    k, v, ks, vs = pools
    NB, bs, Hk, D = k.shape
    pairs = torch.tensor(copies, dtype=torch.int32).cuda()
    binding.pa_copy_blocks(k, v, pairs, len(copies), Hk, D // 2, bs, NB, dtype=binding.PA_BF16)
    binding.pa_copy_blocks(ks, vs, pairs, len(copies), Hk, 1, bs, NB, dtype=binding.PA_F32)


@pytest.mark.parametrize("Hk, D, bs", [(2, 128, 16), (3, 64, 8), (1, 128, 4)])
def test_fork_append_decode(Hk, D, bs):
    rng = np.random.default_rng(Hk)
    H, n, NB = 4 * Hk, 3 * bs + bs // 2, 24
    m = binding.BlockManager(NB, bs, 4, 8)
    pools = [torch.randint(-127, 128, (NB, bs, Hk, D), dtype=torch.int8).cuda() for _ in range(2)]
    pools += [torch.full((NB, Hk, bs), float("nan")).cuda() for _ in range(2)]
    rows = {}

    def write(seq, count):
        slots, copies = m.append(seq, count)
        if copies:
            _copy(pools, copies)
        x = [torch.from_numpy(rng.standard_normal((count, Hk, D), dtype=np.float32)).to(torch.bfloat16) for _ in range(2)]
        binding.write_cache_int8(x[0].cuda(), x[1].cuda(), slots.cuda(), *pools)
        old = rows.get(seq)
        rows[seq] = x if old is None else [torch.cat(p) for p in zip(old, x)]
        return copies

    assert not write(0, n)
    m.fork(0, 1)
    rows[1] = rows[0]
    assert len(write(1, 1)) == 1  # the half-filled block is shared: the child gets its own
    assert not write(0, 3)
    tables, lens = m.export()
    k, v, ks, vs = pools
    q = torch.from_numpy(rng.standard_normal((2, H, D), dtype=np.float32)).to(torch.bfloat16)
    out = binding.decode_int8(q.cuda(), k, v, ks, vs, tables[:2].cuda(), lens[:2].cuda(), D**-0.5)
    for s in (0, 1):
        c = int(lens[s])
        held = []
        for x in rows[s]:
            codes, scale = chunks.quantise(x.float().numpy())
            held.append(codes.astype(np.float64) * scale.astype(np.float64)[..., None])
        pool = [np.zeros((8, bs, Hk, D)) for _ in range(2)]
        for p, x in zip(pool, held):
            p.reshape(-1, Hk, D)[:c] = x
        want, spread, reach = chunks.prefill(q[s : s + 1].double().numpy(), *pool, np.arange(8)[None], np.array([c]),
                                             np.array([0, 1]), D**-0.5, bs)
        # Weights times scales in f16, 2^-11; the exponential and the running sums less than 2^-13; scores as in chunklib.
        room = spread * (2.0**-11 + 2.0**-13 + 2 * (D + 8) * 2.0**-23 * reach)[..., None] + 2.0**-38 * 127 * c * 1.0
        assert_rounded(out[s : s + 1], want, room, 1.0, f"sequence {s}")
    m.close()
