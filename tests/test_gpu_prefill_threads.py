"""Chunk attention and decode over int8 pools without a workspace: from several host threads at once, and on another
stream than the current one."""

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

from chunklib import Chunks
from test_gpu_threads import run_threads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _calls(seed):
    """Functions of a stream: ragged chunks over each type of pool, decode over int8 pools in either of its forms."""
    shapes = [([140, 1, 30], [400, 2000, 0]), ([1, 1, 1, 1], [900, 5, 3000, 64]), ([300], [100]), ([9, 0, 77], [20, 7, 1500])]
    new, old = shapes[seed]
    calls = []
    for pool in ("bf16", "int8", "f32"):
        b = Chunks(new, old, pool, 8, 2, (64, 128)[seed % 2], gap=0, seed=seed)
        calls.append(lambda s, b=b, args=b.gpu(): b.call(args, stream=s))
    for Q in (1, 20):
        b = Chunks([Q] * 3, [seed * 300, 40, 2000], "int8", 8, 2, 128, gap=0, seed=seed)
        q, k, v, ks, vs, tables, lens, _, scale = b.gpu()
        q = q.view(3, Q, 8, 128)
        calls.append(lambda s, a=(q, k, v, ks, vs, tables, lens, scale): binding.decode_int8(*a, stream=s))
    return calls


@pytest.mark.parametrize("one_stream", [True, False])
def test_threads(one_stream):
    calls = [_calls(i) for i in range(4)]
    alone = [[c(None) for c in cs] for cs in calls]
    torch.cuda.synchronize()
    shared = torch.cuda.Stream()
    got = [[] for _ in calls]

    def work(i):
        torch.cuda.set_device(0)
        stream = shared if one_stream else torch.cuda.Stream()
        for n in range(15):
            got[i].append([c(stream) for c in calls[(i + n) % 4]])

    run_threads(work)
    torch.cuda.synchronize()
    for i in range(4):
        for n, outs in enumerate(got[i]):
            for a, b in zip(outs, alone[(i + n) % 4]):
                torch.testing.assert_close(a, b, rtol=0, atol=0)


@pytest.mark.parametrize("raw", [False, True])
def test_work_queued_on_the_current_stream_leaves_the_output_alone(raw):
    for call in _calls(0):
        want = call(None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for _ in range(2):
            late = torch.empty_like(want)
            torch.cuda._sleep(30_000_000)
            late.fill_(7.0)
            del late
            out = call(side.cuda_stream if raw else side)
            torch.cuda.synchronize()
            torch.testing.assert_close(out, want, rtol=0, atol=0)


def test_decode_int8_batches_that_grow():
    """More and more sequences on one stream, with more tickets than its buffer held; then few again."""
    stream = torch.cuda.Stream()
    for S in (3, 2100, 5):
        b = Chunks([1] * S, [(37 * i) % 50 for i in range(S - 1)] + [3000], "int8", 8, 8, 64, gap=0, seed=S)
        q, k, v, ks, vs, tables, lens, _, scale = b.gpu()
        torch.cuda.synchronize()
        out = binding.decode_int8(q, k, v, ks, vs, tables, lens, scale, stream=stream)
        torch.cuda.synchronize()
        b.compare(out, f"{S} sequences")
