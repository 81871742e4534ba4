"""Outputs that the Python layer makes for a call on another stream than the current one: work still queued on the
current stream does not write into them, and they are not handed out again while the current stream reads them."""

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


S, Q, Hk, G, D, bs, n = 5, 2, 2, 4, 64, 16, 6


def _calls():
    gen = torch.Generator().manual_seed(4)
    NB = S * n
    k, v = (torch.randn(NB, bs, Hk, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    k8, v8 = (torch.randint(0, 0x60, (NB, bs, Hk, D), generator=gen, dtype=torch.uint8).cuda() for _ in range(2))
    table = torch.randperm(NB, generator=gen).to(torch.int32).view(S, n)
    table[:, :2] = table[0, :2].clone()
    table = table.cuda()
    prefix = table[0, :2].contiguous()
    lens = torch.full((S,), n * bs - 3, dtype=torch.int32).cuda()
    q = torch.randn(S, Q, G * Hk, D, generator=gen).to(torch.bfloat16).cuda()
    sc = D**-0.5
    return {
        "multi": lambda s: binding.decode_multi(q, k, v, table, lens, sc, stream=s),
        "mod": lambda s: binding.decode_mod(q, k, v, table, lens, sc, stream=s),
        "fp8 mod": lambda s: binding.decode_fp8_mod(q, k8, v8, table, lens, sc, 1.0, 1.0, stream=s),
        "prefix": lambda s: binding.decode_prefix(q, k, v, prefix, table, lens, sc, stream=s),
        "fp8 prefix": lambda s: binding.decode_fp8_prefix(q, k8, v8, prefix, table, lens, sc, 1.0, 1.0, stream=s),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["multi", "mod", "fp8 mod", "prefix", "fp8 prefix"])
def test_work_queued_on_the_current_stream_leaves_the_output_alone(name, raw):
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        # Memory of the output's size, freed with a write to it still queued behind a delay.
        late = torch.empty_like(want)
        torch.cuda._sleep(30_000_000)
        late.fill_(7.0)
        del late
        out = call(side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_tables_step():
    tables = torch.full((S, n), -1, dtype=torch.int32, device="cuda")
    new = torch.tensor([3, 0, 20, 1, 16], dtype=torch.int32, device="cuda")
    zero = torch.zeros(S, dtype=torch.int32, device="cuda")
    free, count = torch.arange(64, dtype=torch.int32, device="cuda"), torch.tensor([64], dtype=torch.int32, device="cuda")
    slots = torch.empty(64, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late = [torch.empty(S, dtype=torch.int32, device="cuda") for _ in range(3)]
    torch.cuda._sleep(30_000_000)
    for x in late:
        x.fill_(99)
    del late, x
    lens, left, starts = binding.tables_step(tables, zero, new, free, count, bs, slots, stream=side)
    torch.cuda.synchronize()
    assert lens.tolist() == new.tolist()
    assert left.tolist() == [64 - 5]
    assert starts.tolist() == [0, 3, 3, 23, 24, 40]


def test_the_current_streams_reads_come_before_the_memory_is_used_again():
    call = _calls()["mod"]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(30_000_000)
    copy = out.clone()  # queued behind the delay
    del out
    with torch.cuda.stream(side):
        other = torch.full_like(want, 5.0)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and (other == 5).all()
