"""Decode calls of different shapes in one workspace: every call finds its merge tickets at zero."""

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


class Batch:
    """S sequences of Q queries over a pool of `kind` with tokens of lo .. hi, drawn on the device."""

    def __init__(self, kind, S, Q, lo, hi, num_ranges=0, heads=32, kv_heads=8, D=128, bs=16):
        g = torch.Generator(device="cuda").manual_seed(S * 7 + Q)
        self.kind, self.num_ranges = kind, num_ranges
        self.shape = (S, Q, heads, kv_heads, D, num_ranges)
        self.lens = torch.randint(lo, hi + 1, (S,), generator=g, device="cuda", dtype=torch.int32)
        width = (hi + bs - 1) // bs
        blocks = S * width + 1
        self.tables = torch.randperm(blocks, generator=g, device="cuda")[: S * width].to(torch.int32).view(S, width)
        pool = (blocks, bs, kv_heads, D)
        if kind == "int8":
            self.pools = [torch.randint(-127, 128, pool, generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
            self.pools += [torch.rand(blocks, kv_heads, bs, generator=g, device="cuda") / 64 for _ in range(2)]
        else:
            self.pools = [torch.randn(pool, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
            if kind == "fp8":
                self.pools = [p.to(torch.float8_e4m3fn).view(torch.uint8) for p in self.pools]
        self.q = torch.randn(S, Q, heads, D, generator=g, device="cuda").to(torch.bfloat16)

    def size(self):
        S, Q, heads, kv_heads, D, R = self.shape
        of = binding.pa_decode_int8_workspace_size if self.kind == "int8" else binding.pa_decode_mq_workspace_size
        return of(S, Q, heads, kv_heads, D, R)

    def call(self, ws):
        out = torch.full_like(self.q, float("nan"))
        kw = dict(out=out, workspace=ws, num_ranges=self.num_ranges)
        scale = self.shape[4] ** -0.5
        if self.kind == "int8":
            return binding.decode_int8(self.q, *self.pools, self.tables, self.lens, scale, **kw)
        if self.kind == "fp8":
            return binding.decode_fp8_multi(self.q, *self.pools, self.tables, self.lens, scale, 1.0, 1.0, **kw)
        return binding.decode_multi(self.q, *self.pools, self.tables, self.lens, scale, **kw)


def _in_turns(batches, order, slices):
    """The batches in one buffer one after another, against each in a fresh one."""
    want = [b.call(torch.zeros(b.size(), dtype=torch.uint8, device="cuda")) for b in batches]
    assert all(bool(torch.isfinite(w).all()) for w in want)
    ws = torch.zeros(max(b.size() for b in batches), dtype=torch.uint8, device="cuda")
    for i in order:
        b = batches[i]
        got = b.call(ws[: b.size()] if slices else ws)
        assert torch.equal(got, want[i]), f"batch {i} of {order}"


@pytest.mark.parametrize("slices", [False, True])
@pytest.mark.parametrize("kind", ["int8", "bf16", "fp8"])
def test_shapes_share_a_buffer(kind, slices):
    """Few sequences of several queries, many of one, and a call of more ranges than tickets have room for."""
    batches = [Batch(kind, 4, 2, 3000, 3100), Batch(kind, 1033, 1, 20, 60), Batch(kind, 1300, 1, 20, 60),
               Batch(kind, 4, 2, 3000, 3100, num_ranges=700)]
    _in_turns(batches, [0, 1, 0, 2, 3, 2, 3, 1, 0], slices)


@pytest.mark.parametrize("slices", [False, True])
def test_shapes_that_run_as_chunks_share_it_too(slices):
    """Shapes that the decode kernel does not take leave its tickets alone."""
    batches = [Batch("int8", 3, 5, 2000, 2100, heads=64), Batch("int8", 4300, 1, 10, 40),
               Batch("int8", 2, 1, 900, 1000, heads=4, kv_heads=1, D=64), Batch("int8", 5, 1, 700, 3000, heads=16, D=64)]
    _in_turns(batches, [0, 1, 2, 3, 0, 3, 2, 1], slices)


@pytest.mark.parametrize("num_ranges", [513, 514, 4096])
def test_many_ranges_in_a_buffer_of_any_content(num_ranges):
    """513 ranges of 8 KV heads have their tickets in the room at the buffer's start; those of more are cleared."""
    b = Batch("bf16", 3, 1, 6000, 9000, num_ranges)
    want = b.call(torch.zeros(b.size(), dtype=torch.uint8, device="cuda"))
    ws = torch.full((b.size(),), 255, dtype=torch.uint8, device="cuda")
    ws[:16384] = 0
    for _ in range(2):
        assert torch.equal(b.call(ws), want)
    graph_out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graph_out.copy_(b.call(ws))
    ws[16384:] = 255
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(graph_out, want)


def _others(b):
    """(size, call) of what takes scratch of any content, over a bf16 batch's pools."""
    S, Q, H, Hk, D, _ = b.shape
    k, v = b.pools
    starts = torch.arange(S + 1, device="cuda", dtype=torch.int32) * Q
    scale = D**-0.5
    codes = [(30 * x).clamp(-127, 127).to(torch.int8) for x in (k, v)]
    scales = [torch.full((k.shape[0], Hk, k.shape[1]), 1 / 30, device="cuda") for _ in range(2)]
    fp8 = [x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v)]
    tables = b.tables.clone()
    tables[:, :2] = tables[0, :2]
    rows = b.q.view(S * Q, H, D)
    chunk, mod = binding.pa_prefill_workspace_size(D), binding.pa_decode_mod_workspace_size
    prefix = binding.pa_decode_prefix_workspace_size(S, Q, H, Hk, D)
    return {
        "prefill": (chunk, lambda ws: binding.prefill(rows, k, v, b.tables, b.lens, starts, scale, workspace=ws)),
        "prefill f32": (chunk, lambda ws: binding.prefill(rows.float(), k.float(), v.float(), b.tables, b.lens, starts, scale,
                                                          workspace=ws)),
        "prefill int8": (chunk, lambda ws: binding.prefill_int8(rows, *codes, *scales, b.tables, b.lens, starts, scale,
                                                                workspace=ws)),
        "mod": (mod(S, Q, H, Hk, D, binding.PA_BF16),
                lambda ws: binding.decode_mod(b.q, k, v, b.tables, b.lens, scale, softcap=20.0, workspace=ws)),
        "fp8 mod": (mod(S, Q, H, Hk, D, binding.PA_FP8_E4M3),
                    lambda ws: binding.decode_fp8_mod(b.q, *fp8, b.tables, b.lens, scale, 1.0, 1.0, window=900, workspace=ws)),
        "prefix": (prefix, lambda ws: binding.decode_prefix(b.q, k, v, tables[0, :2].contiguous(), tables, b.lens, scale,
                                                            workspace=ws)),
        "fp8 prefix": (prefix, lambda ws: binding.decode_fp8_prefix(b.q, *fp8, tables[0, :2].contiguous(), tables, b.lens,
                                                                    scale, 1.0, 1.0, workspace=ws)),
    }


@pytest.mark.parametrize("other", ["prefill", "prefill f32", "prefill int8", "mod", "fp8 mod", "prefix", "fp8 prefix"])
def test_kinds_of_calls_share_a_buffer(other):
    """A decode's tickets survive calls whose scratch may hold anything, before and behind it in one buffer."""
    decodes = [Batch("bf16", 4, 2, 3000, 3100), Batch("int8", 300, 1, 20, 600), Batch("fp8", 3, 4, 500, 4000)]
    size, call = _others(Batch("bf16", 5, 2, 900, 2000))[other]
    fresh = lambda n: torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
    want = call(fresh(size)).clone()
    wants = [d.call(torch.zeros(d.size(), dtype=torch.uint8, device="cuda")) for d in decodes]
    ws = torch.zeros(max(size, *(d.size() for d in decodes)), dtype=torch.uint8, device="cuda")
    for slices in (False, True):
        for d, w in zip(decodes, wants):
            assert torch.equal(call(ws[:size] if slices else ws), want)
            assert torch.equal(d.call(ws[: d.size()] if slices else ws), w)
    with pytest.raises(binding.PagedAttnError) as e:
        call(ws[: size // 64 // 256 * 256])
    assert e.value.code == binding.PA_ERR_WORKSPACE
