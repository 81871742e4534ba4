"""GPU parity of decode with modified scores (pa_decode_mod, pa_decode_fp8_mod)
against its fp64 restatement.

Bounds, as relative errors of a softmax weight: the scores are fp32 sums of D
products of magnitude ~1 (D <= 128 roundings of 2^-24 of a partial sum below
2^4 times the scale), so 2^-13 covers them, the cap's 2^-23 * 50 and the SFU's
2^x (2^-22) on both sides of the division.  FP8 pools: the weights enter the
product rounded to f16, 2^-11 more.  fp32 pools add their shorter sums (4
products and 5 additions): 2^-15.  The output's own rounding comes on top."""

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle import modified
from paged_kv_cache_292_gb300 import binding, workloads

from paritylib import assert_rounded, captured, refused_under_capture

pytestmark = pytest.mark.gpu

WEIGHT_ERROR = {"bf16": 2.0**-13, "fp8": 2.0**-13 + 2.0**-11, "f32": 2.0**-15}
KS, VS = 0.02, 0.015


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


class Batch:
    """A seeded batch whose unseen tokens are NaN in the pool and whose unseen blocks have no table entry."""

    def __init__(self, dtype, ctx, Q=1, heads=8, kv_heads=2, D=128, bs=16, seed=0, **mods):
        self.dtype, self.Q, self.bs, self.mods = dtype, Q, bs, mods
        ctx = np.asarray(ctx)
        S = len(ctx)
        sp = workloads.spec("llama3_8b", num_seqs=S, num_heads=heads, num_kv_heads=kv_heads, head_size=D,
                            block_size=bs, max_context=int(ctx.max()) + 3 * bs, pool_blocks=0, seed=seed,
                            dtype="f32" if dtype == "f32" else "bf16")
        w = workloads.make_workload(sp, prewritten=True, poison=True, context_lens=ctx)
        q = np.random.default_rng([seed, 78]).standard_normal((S, Q, heads, D), dtype=np.float32)
        self.q = torch.from_numpy(q).to(w.q.dtype)
        self.ctx, self.tables, self.scale, self.S = ctx, w.block_tables.numpy().copy(), w.scale, S
        pools = [w.k_cache, w.v_cache]
        if dtype == "fp8":
            pools = [torch.from_numpy(np.where(np.isnan(x.float().numpy()), 0x7F,
                                               ofp8.quantize(np.nan_to_num(x.float().numpy()), sc)).astype(np.uint8))
                     for x, sc in zip(pools, (KS, VS))]
        nan = 0x7F if dtype == "fp8" else float("nan")
        for s, c in enumerate(ctx.tolist()):
            seen = modified.seen_by_some(c, Q, mods.get("window", 0), self._of("first", s), self._of("prefix", s))
            for t in np.flatnonzero(~seen):
                for x in pools:
                    x[int(w.block_tables[s, t // bs]), t % bs] = nan
            hidden = np.ones(self.tables.shape[1], dtype=bool)
            hidden[np.flatnonzero(seen) // bs] = False
            self.tables[s, hidden] = -1
        self.k, self.v = pools

    def _of(self, name, s):
        x = self.mods.get(name)
        return 0 if x is None else int(x[s])

    def want(self):
        k, v = (x.double().numpy() for x in (self.k, self.v)) if self.dtype != "fp8" else (
            ofp8.e4m3_decode(x.numpy()) * float(np.float32(sc)) for x, sc in ((self.k, KS), (self.v, VS)))
        return modified.decode_mod(self.q.double().numpy(), k, v, self.tables, self.ctx, self.scale, self.bs,
                                   **self.mods)

    def gpu(self):
        i32 = lambda x: None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
        m = self.mods
        q = self.q.cuda() if self.Q > 1 else self.q[:, 0].contiguous().cuda()
        args = (q, self.k.cuda(), self.v.cuda(), i32(self.tables), i32(self.ctx), self.scale)
        slopes = m.get("slopes")
        kw = dict(softcap=m.get("softcap", 0.0), window=m.get("window", 0), first_tokens=i32(m.get("first")),
                  prefix_lens=i32(m.get("prefix")),
                  alibi_slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda())
        return args, kw

    def call(self, args, kw, **more):
        if self.dtype == "fp8":
            return binding.decode_fp8_mod(*args, KS, VS, **kw, **more)
        return binding.decode_mod(*args, **kw, **more)

    def check(self, what, **more):
        args, kw = self.gpu()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(args[0], float("nan"))
        self.call(args, kw, out=out, error_flag=err, check_block_ids=True, **more)
        torch.cuda.synchronize()
        assert int(err) == 0
        want, spread = self.want()
        assert_rounded(out.view(self.S, self.Q, *out.shape[-2:]), want, spread, WEIGHT_ERROR[self.dtype], what)
        return out


def _slopes(heads):
    return np.float32(2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)).astype(np.float64)


CTX = [1, 2, 15, 16, 17, 33, 100, 257, 400, 3, 64, 31]
S = len(CTX)
RNG = np.random.default_rng(3)
MODS = {
    "plain": dict(),
    "cap": dict(softcap=2.0),
    "alibi": dict(alibi=True),
    "window 1": dict(window=1),
    "window 7": dict(window=7),
    "window 16": dict(window=16, softcap=30.0),
    "window 100": dict(window=100, alibi=True),
    "window beyond": dict(window=2**31 - 1),
    "first": dict(first=RNG.integers(-3, 60, S)),
    "first at the end": dict(first=np.array(CTX) - 1),
    "first behind the end": dict(first=np.array(CTX) + 2),
    "first far behind": dict(first=[2**31 - 1] * S),
    "prefix": dict(prefix=RNG.integers(-3, 60, S)),
    "prefix is all": dict(prefix=[2**31 - 1] * S, softcap=5.0),
    "prefix and window": dict(prefix=RNG.integers(0, 40, S), window=20),
    "prefix far from window": dict(prefix=[5] * S, window=3, alibi=True),
    "all": dict(prefix=RNG.integers(0, 90, S), window=33, first=RNG.integers(0, 30, S), alibi=True, softcap=3.0),
}


def _mods(name, heads):
    m = dict(MODS[name])
    if m.pop("alibi", False):
        m["slopes"] = _slopes(heads)
    return m


@pytest.mark.parametrize("name", MODS)
@pytest.mark.parametrize("dtype, Q, heads, kv_heads, D", [
    ("bf16", 1, 8, 2, 128), ("bf16", 2, 8, 2, 64), ("bf16", 5, 12, 3, 128), ("bf16", 4, 16, 2, 64),
    ("fp8", 1, 8, 2, 128), ("fp8", 3, 14, 2, 64), ("fp8", 2, 3, 3, 128), ("f32", 1, 4, 2, 64), ("f32", 1, 8, 1, 128),
    ("f32", 1, 3, 1, 128)])
def test_masks_and_types(name, dtype, Q, heads, kv_heads, D):
    Batch(dtype, CTX, Q, heads, kv_heads, D, **_mods(name, heads)).check(f"{name} {dtype} Q={Q}")


@pytest.mark.parametrize("bs", [1, 5, 8, 24, 32, 256])
@pytest.mark.parametrize("dtype, Q", [("bf16", 1), ("bf16", 3), ("fp8", 2), ("f32", 1)])
@pytest.mark.parametrize("name", ["all", "prefix far from window"])
def test_block_sizes(bs, dtype, Q, name):
    Batch(dtype, CTX, Q, 8, 2, 128, bs, **_mods(name, 8)).check(f"bs={bs}")


@pytest.mark.parametrize("num_ranges", [1, 2, 13, 997])
@pytest.mark.parametrize("dtype, Q", [("bf16", 1), ("bf16", 4), ("fp8", 4), ("f32", 1)])
def test_cut_sequences(num_ranges, dtype, Q):
    Batch(dtype, CTX, Q, **_mods("all", 8)).check(f"R={num_ranges}", num_ranges=num_ranges)


@pytest.mark.parametrize("dtype, Q", [("bf16", 1), ("fp8", 2)])
def test_long_context_with_a_far_prefix(dtype, Q):
    """The walk jumps over more table entries than its window of the table holds."""
    ctx = [9000, 40, 5003]
    Batch(dtype, ctx, Q, 4, 2, 64, 8, prefix=[20, 9, 700], window=50).check("far prefix")


def test_empty_sequences_and_queries_before_the_start():
    ctx = [0, 1, 0, 2, 40, 3, 0]
    for dtype in ("bf16", "fp8"):
        out = Batch(dtype, ctx, 4, prefix=[9] * 7, window=2).check("short")
        assert torch.all(out[0] == 0) and torch.all(out[1, :3] == 0) and torch.all(out[3, :2] == 0)


def test_large_scores():
    """Dot products near 2^90 become +-cap."""
    b = Batch("bf16", [40, 7], 1, softcap=4.0)
    b.q *= 2.0**60
    b.k = b.k.clone() * 2.0**30
    args, kw = b.gpu()
    out = b.call(args, kw)
    want, spread = b.want()
    assert_rounded(out[:, None], want, spread, WEIGHT_ERROR["bf16"], "large scores")


def test_bad_block_id_of_a_seen_block_is_reported():
    b = Batch("bf16", [100, 50], 1, window=20)
    args, kw = b.gpu()
    args[3][0, 6] = 10**6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.call(args, kw, error_flag=err, check_block_ids=True)
    assert int(err) == binding.PA_DEVERR_BLOCK_ID


@pytest.mark.parametrize("dtype, Q", [("bf16", 1), ("bf16", 5), ("fp8", 5), ("f32", 1)])
def test_workspace_of_any_content_capture_and_streams(dtype, Q):
    """A caller's scratch filled with ones, shared by two captured graphs of different shapes on one stream."""
    a = Batch(dtype, CTX, Q, **_mods("all", 8))
    b = Batch(dtype, [700, 5], Q, seed=4, **dict(window=300))
    kv = {"f32": binding.PA_F32, "bf16": binding.PA_BF16, "fp8": binding.PA_FP8_E4M3}[dtype]
    size = binding.pa_decode_mod_workspace_size(S, Q, 8, 2, 128, kv)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    parts = [(x, *x.gpu()) for x in (a, b)]
    outs = [torch.full_like(args[0], float("nan")) for _, args, _ in parts]
    graphs = []
    for (x, args, kw), out in zip(parts, outs):
        # Scratch of the library's own does not go into a graph.
        assert refused_under_capture(lambda: x.call(args, kw, out=out), binding.PagedAttnError)
        graphs.append(captured(lambda: x.call(args, kw, out=out, workspace=ws)))
    for _ in range(2):
        for g in graphs:
            g.replay()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    eager = [x.call(args, kw, stream=side) for x, args, kw in parts]
    torch.cuda.synchronize()
    for (x, _, _), out, e in zip(parts, outs, eager):
        want, spread = x.want()
        assert_rounded(out.view(want.shape), want, spread, WEIGHT_ERROR[dtype], "captured")
        assert torch.equal(out, e)
    with pytest.raises(binding.PagedAttnError) as err:
        a.call(*parts[0][1:], workspace=ws[: size // 64 // 256 * 256])
    assert err.value.code == binding.PA_ERR_WORKSPACE


def test_plain_modification_equals_decode():
    b = Batch("bf16", CTX, 1)
    args, kw = b.gpu()
    want, spread = b.want()
    for got in (b.call(args, kw, num_ranges=1), b.call(args, kw)):
        assert_rounded(got, binding.decode(*args).double().cpu().numpy(), spread[:, 0], WEIGHT_ERROR["bf16"] + 2.0**-8,
                       "against decode")


def test_python_layer_refuses_mismatched_arguments():
    b = Batch("bf16", CTX, 1)
    args, kw = b.gpu()
    q, k, v, tables, lens, scale = args
    bad = [
        dict(alibi_slopes=torch.zeros(7, device="cuda")),
        dict(alibi_slopes=torch.zeros(8, dtype=torch.float64, device="cuda")),
        dict(first_tokens=lens[:-1].contiguous()),
        dict(prefix_lens=lens.long()),
    ]
    for m in bad:
        with pytest.raises(ValueError):
            binding.decode_mod(*args, **m)
    for other in ((q[:-1].contiguous(), k, v, tables, lens), (q, k[:, :, :, :64].contiguous(), v, tables, lens),
                  (q, k, v, tables.long(), lens), (q.float(), k, v, tables, lens), (q[:, ::2], k, v, tables, lens)):
        with pytest.raises(ValueError):
            binding.decode_mod(*other, scale)


@pytest.mark.parametrize("cap", [1e-40, 1e-3, 40.0, 1e3, 1e6, 1e20, 3e38])
@pytest.mark.parametrize("dtype, Q", [("bf16", 1), ("bf16", 4), ("bf16", 5), ("fp8", 1), ("fp8", 5), ("f32", 1)])
def test_caps_of_every_size(cap, dtype, Q):
    """The smallest caps make all scores alike, the largest change none.  Caps up to 64 add 2^-22 of the cap,
    larger ones 2^-19 of a score at most, or where it is below an eighth of the cap 2^-23 of it."""
    Batch(dtype, [1, 70, 300], Q, softcap=cap).check(f"cap {cap} {dtype} Q={Q}")


@pytest.mark.parametrize("dtype, Q", [("bf16", 1), ("fp8", 5), ("f32", 1)])
def test_calls_on_many_streams_at_once(dtype, Q):
    """The library's scratch is one buffer per stream: calls that overlap do not meet in it, also beyond the
    number of streams it keeps buffers for."""
    parts = [Batch(dtype, ctx, Q, seed=i, window=w) for i, (ctx, w) in enumerate([([3000, 9], 0), ([1500, 2000], 700)])]
    calls = [(x, *x.gpu()) for x in parts]
    wants = [x.call(args, kw) for x, args, kw in calls]
    streams = [torch.cuda.Stream() for _ in range(11)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for j in range(4):
            got += [(i, x.call(args, kw, stream=st)) for k, st in enumerate(streams[:2 if j < 3 else 11])
                    for i, (x, args, kw) in enumerate(calls) if i == (j + k) % 2]
        torch.cuda.synchronize()
        for i, out in got:
            assert torch.equal(out, wants[i])
