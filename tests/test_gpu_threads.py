"""Calls without a workspace from several host threads at once: on one stream with batches that grow, and on more
streams than the library keeps buffers for.  Every result is that of the same call made alone."""

import threading

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

pytestmark = pytest.mark.gpu

Hk, G, D, bs, P = 2, 4, 64, 16, 12


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


class Batch:
    def __init__(self, S, seed):
        gen = torch.Generator().manual_seed(seed)
        nblk = P + 3
        NB = P + 3 * S
        self.pools = [torch.randn(NB, bs, Hk, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
        own = P + torch.randperm(3 * S, generator=gen).view(S, 3)
        self.prefix = torch.arange(P, dtype=torch.int32).cuda()
        self.table = torch.cat([torch.arange(P).expand(S, -1), own], 1).to(torch.int32).contiguous().cuda()
        self.lens = (P * bs + torch.randint(1, 3 * bs + 1, (S,), generator=gen)).to(torch.int32).cuda()
        self.q = torch.randn(S, G * Hk, D, generator=gen).to(torch.bfloat16).cuda()
        assert self.table.shape[1] == nblk

    def calls(self, stream=None):
        args = (self.q, *self.pools)
        rest = (self.table, self.lens, D**-0.5)
        return [binding.decode_prefix(*args, self.prefix, *rest, stream=stream),
                binding.decode_mod(*args, *rest, stream=stream, softcap=20.0, window=100)]


def run_threads(work):
    errors = []

    def guarded(i):
        try:
            work(i)
        except BaseException as e:  # noqa: BLE001 - reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("sizes", [(9, 9, 9, 9), (3, 40, 150, 500)])
def test_one_stream(sizes):
    batches = [Batch(S, seed) for seed, S in enumerate(sizes)]
    alone = [b.calls() for b in batches]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = [[] for _ in batches]

    def work(i):
        torch.cuda.set_device(0)
        for n in range(30):
            got[i].append(batches[(i + n) % 4].calls(stream))

    run_threads(work)
    torch.cuda.synchronize()
    for i in range(4):
        for n, outs in enumerate(got[i]):
            for a, b in zip(outs, alone[(i + n) % 4]):
                assert torch.equal(a, b)


def test_eleven_streams():
    batches = [Batch(S, seed) for seed, S in enumerate((5, 64, 9, 200))]
    alone = [b.calls() for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(11)]
    got = [[] for _ in batches]

    def work(i):
        torch.cuda.set_device(0)
        for n in range(22):
            got[i].append(batches[(i + n) % 4].calls(streams[(3 * i + n) % 11]))

    run_threads(work)
    torch.cuda.synchronize()
    for i in range(4):
        for n, outs in enumerate(got[i]):
            for a, b in zip(outs, alone[(i + n) % 4]):
                assert torch.equal(a, b)
