"""A decode call whose copy is withheld leaves every merge ticket at zero: the next call is right without the scratch
being cleared, the library's own (which a caller cannot clear) and a caller's."""

import time

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

pytestmark = pytest.mark.gpu

KINDS = {"f32": (torch.float32, 1), "bf16": (torch.bfloat16, 1), "mq": (torch.bfloat16, 2), "split": (torch.bfloat16, 5),
         "fp8": (torch.uint8, 1), "fp8 split": (torch.uint8, 8), "int8": (torch.int8, 1), "int8 mq": (torch.int8, 2),
         "int8 split": (torch.int8, 7)}
H, HK, D, BS = 8, 2, 128, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


class Step:
    def __init__(self, kind, lens):
        pool, self.Q = KINDS[kind]
        g = torch.Generator(device="cuda").manual_seed(len(lens))
        self.kind, self.lens = kind, torch.tensor(lens, dtype=torch.int32, device="cuda")
        width = (max(lens) + BS - 1) // BS
        blocks = len(lens) * width
        self.tables = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).view(len(lens), width)
        x = [torch.randn(blocks, BS, HK, D, generator=g, device="cuda") for _ in range(2)]
        if pool is torch.int8:
            self.pools = [(40 * p).clamp(-127, 127).to(pool) for p in x]
            self.pools += [torch.rand(blocks, HK, BS, generator=g, device="cuda") / 32 for _ in range(2)]
        elif pool is torch.uint8:
            self.pools = [p.to(torch.float8_e4m3fn).view(pool) for p in x]
        else:
            self.pools = [p.to(pool) for p in x]
        self.q = torch.randn(len(lens), self.Q, H, D, generator=g, device="cuda").to(
            torch.float32 if kind == "f32" else torch.bfloat16)

    def call(self, **kw):
        out = torch.full_like(self.q, float("nan"))
        q, o = (self.q, out) if self.Q > 1 else (self.q[:, 0], out[:, 0])
        args = (*self.pools, self.tables, self.lens, D**-0.5)
        if self.kind.startswith("int8"):
            binding.decode_int8(q, *args, out=o, **kw)
        elif self.kind.startswith("fp8"):
            binding.decode_fp8_multi(self.q, *args, 1.0, 1.0, out=out, **kw)
        elif self.Q > 1:
            binding.decode_multi(q, *args, out=o, **kw)
        else:
            binding.decode(q, *args, out=o, **kw)
        torch.cuda.synchronize()
        return out


def _withheld_then_again(step, want, tile, **kw):
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.pa_test_stall_copy(tile, 1000)
    t0 = time.perf_counter()
    step.call(error_flag=flag, **kw)
    assert time.perf_counter() - t0 < 0.5
    assert int(flag) == binding.PA_DEVERR_TIMEOUT
    flag.zero_()
    assert torch.equal(step.call(error_flag=flag, **kw), want)
    assert int(flag) == 0


def _tiles(lens):
    return sum(-(-c // 16) for c in lens)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("lens", [[3000, 40, 9, 5000, 700], [20000], [20] * 150 + [9000] + [33] * 200], ids=["few", "one", "many"])
def test_tickets_after_a_timeout(kind, lens):
    step = Step(kind, lens)
    want = step.call()
    size = (binding.pa_decode_int8_workspace_size if kind.startswith("int8") else binding.pa_decode_mq_workspace_size)
    ws = torch.zeros(size(len(lens), step.Q, H, HK, D), dtype=torch.uint8, device="cuda")
    assert torch.equal(step.call(workspace=ws), want)
    total = _tiles(lens)
    for tile in (0, 1, total // 3, total // 2, total - 2, total - 1):
        _withheld_then_again(step, want, tile)
        _withheld_then_again(step, want, tile, workspace=ws)
        assert int(ws[:16384].view(torch.int32).abs().sum()) == 0


@pytest.mark.parametrize("num_ranges", [2, 5, 40, 600])
def test_tickets_of_forced_ranges(num_ranges):
    lens = [600, 1, 16, 17, 900, 300, 2500]
    for kind in ("bf16", "int8"):
        step = Step(kind, lens)
        want = step.call(num_ranges=num_ranges)
        for tile in range(0, _tiles(lens), 23):
            _withheld_then_again(step, want, tile, num_ranges=num_ranges)


def test_a_timeout_on_one_stream_and_calls_on_many():
    """The scratch of a stream that timed out passes to other streams, of which there are more than kept buffers."""
    step = Step("int8", [4000, 100, 2000])
    want = step.call()
    streams = [torch.cuda.Stream() for _ in range(12)]
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _withheld_then_again(step, want, 40 + 7 * i)
    for s in streams[::-1]:
        with torch.cuda.stream(s):
            assert torch.equal(step.call(), want)
