"""GPU parity of decode over a shared prefix in FP8 pools (pa_decode_fp8_prefix)
against the fp64 restatement of multi-query decode on the decoded pools.

Bound: the weights are rounded to f16 (half a step, 2^-11) before they meet V,
scores and exponentials add less than 2^-13 to each weight, and the output is
rounded once.  The queries are exact in f16 (|q| well inside [2^-14, 65504]; a
smaller one is off by 2^-25, which moves no score by 2^-20)."""

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle import modified
from paged_kv_cache_292_gb300 import binding

import test_gpu_prefix as bf16
from paritylib import assert_rounded, captured, refused_under_capture
from test_gpu_prefix import NONE, _lib  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu

WEIGHT_ERROR = 2.0**-11 + 2.0**-13
VS = 0.015


class Batch(bf16.Batch):
    """The bf16 batch with its pools quantised; a pool row without a token holds the NaN code."""

    def __init__(self, *args, spread=1.0, **kw):
        super().__init__(*args, spread=spread, **kw)
        self.ks = 0.02 * max(spread, 0.01)
        self.k, self.v = (self._codes(x, sc) for x, sc in ((self.k, self.ks), (self.v, VS)))

    @staticmethod
    def _codes(x, scale):
        x = x.float().numpy()
        return torch.from_numpy(np.where(np.isnan(x), 0x7F, ofp8.quantize(np.nan_to_num(x), scale)).astype(np.uint8))

    def want(self):
        k, v = (np.nan_to_num(ofp8.e4m3_decode(x.numpy())) * float(np.float32(sc))
                for x, sc in ((self.k, self.ks), (self.v, VS)))
        return modified.decode_mod(self.q.double().numpy(), k, v, self.full, self.ctx, self.scale, self.bs)

    def call(self, args, **kw):
        return binding.decode_fp8_prefix(*args, self.ks, VS, **kw)

    def check(self, what, **kw):
        args = self.gpu()
        out = torch.full_like(args[0], float("nan"))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.call(args, out=out, error_flag=err, check_block_ids=True, **kw)
        torch.cuda.synchronize()
        assert int(err) == 0
        want, spread = self.want()
        assert_rounded(out.view(want.shape), want, spread, WEIGHT_ERROR, what)
        return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads, kv_heads, Q", [(8, 2, 1), (14, 2, 1), (8, 4, 3), (16, 2, 4), (4, 4, 2)])
@pytest.mark.parametrize("blocks", [1, 8, 20, 41])
def test_heads_and_queries(D, heads, kv_heads, Q, blocks):
    Batch(blocks, [Q, Q + 1, 40, 7 + Q, 130], Q, heads, kv_heads, D).check("heads")


@pytest.mark.parametrize("heads, kv_heads, Q", [(3, 3, 1), (8, 1, 1), (5, 1, 6)])
def test_odd_numbers_of_heads(heads, kv_heads, Q):
    Batch(9, [Q, 40, 130], Q, heads, kv_heads, 128).check("odd heads")
    with pytest.raises(binding.PagedAttnError) as e:
        Batch(9, [Q, 40], Q, heads, kv_heads, 64).check("refused")
    assert e.value.code == binding.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("bs", [8, 16, 24, 40, 128, 256])
@pytest.mark.parametrize("tokens", [8, 128, 136, 500])
@pytest.mark.parametrize("D", [64, 128])
def test_block_and_prefix_sizes(bs, tokens, D):
    Batch(max(1, tokens // bs), [1, 30, 2, 65], 1, 8, 2, D, bs).check(f"bs={bs}")


@pytest.mark.parametrize("S", [1, 31, 32, 33, 64, 65, 97, 130])
def test_numbers_of_rows(S):
    """Rows per KV head around one, two and three tiles of 128 (group 4)."""
    Batch(9, (np.arange(S) * 7) % 23 + 1, 1, 8, 2, 64, 16, seed=S).check(f"S={S}")
    Batch(9, (np.arange(S) * 7) % 23 + 1, 1, 8, 2, 128, 16, seed=S).check(f"S={S}")


@pytest.mark.parametrize("Q", [1, 4])
def test_sequences_that_do_not_reach_the_prefixs_end(Q):
    out = Batch(8, [NONE, 5, -3, 0, Q - 1, Q, -100, NONE, 40, Q - 2], Q, 8, 2, 128).check("short")
    assert torch.all(out[0] == 0) and torch.all(out[7] == 0)


def test_no_prefix():
    Batch(0, [5, 17, 1, 100], 1, 8, 2, 128).check("none")
    Batch(0, [5, 17, 3, 100], 3, 8, 2, 64).check("none")


@pytest.mark.parametrize("spread", [0.0, 6.0, 40.0])
def test_flat_and_peaked_scores(spread):
    Batch(40, [3, 50, 200], 1, 8, 2, 128, seed=3, spread=spread).check("spread")


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_scales(scale):
    Batch(20, [3, 50, 200], 1, 8, 2, 128, seed=4, scale=scale).check("scale")


def test_long_prefix_of_small_batch():
    Batch(1100, [3, 50], 1, 4, 2, 64, 8).check("long")


def test_bad_prefix_block_is_reported():
    b = Batch(30, [4, 9, 77], 1, 8, 2, 128)
    b.tables[:, :30] = b.full[:, :30]
    for bad in (-1, b.k.shape[0], 2**31 - 1):
        args = b.gpu()
        args[3][7] = bad
        args[4][:, 7] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        b.call(args, error_flag=err, check_block_ids=True)
        assert int(err) == binding.PA_DEVERR_BLOCK_ID


def test_workspace_of_any_content_capture_and_streams():
    """A caller's scratch filled with ones, shared by graphs of both pool types on one stream."""
    b, plain = Batch(30, np.arange(50) % 7 + 1, 1, 8, 2, 128), bf16.Batch(9, [5, 6], 4, 16, 2, 64)
    size = max(binding.pa_decode_prefix_workspace_size(x.S, x.Q, x.q.shape[2], x.k.shape[2], x.D) for x in (b, plain))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    args, other = b.gpu(), plain.gpu()
    out = torch.full_like(args[0], float("nan"))
    assert refused_under_capture(lambda: b.call(args), binding.PagedAttnError)
    graphs = [captured(lambda: b.call(args, out=out, workspace=ws)),
              captured(lambda: binding.decode_prefix(*other, workspace=ws))]
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    eager = b.call(args, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    want, spread = b.want()
    assert_rounded(out.view(want.shape), want, spread, WEIGHT_ERROR, "captured")
    assert torch.equal(out, eager)


@pytest.mark.parametrize("D, S", [(128, 10), (64, 60), (128, 90)])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_withheld_copy_times_out_and_the_next_call_is_clean(D, S, where):
    b = Batch(32, [3] * S, 1, 8, 2, D)
    args = b.gpu()
    ws = torch.full((binding.pa_decode_prefix_workspace_size(S, 1, 8, 2, D),), 255, dtype=torch.uint8, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = b.call(args, workspace=ws, error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0
    tiles = 4 * 2 * -(-S * 4 // 256)
    binding.pa_test_stall_copy(min(int(where * tiles), tiles - 1), 1000)
    b.call(args, workspace=ws, error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == binding.PA_DEVERR_TIMEOUT
    flag.zero_()
    out = b.call(args, workspace=ws, error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0 and torch.equal(out, ref)


def test_python_layer_refuses_mismatched_arguments():
    b = Batch(8, [5, 6], 1, 8, 2, 64)
    q, k, v, prefix, tables, lens, scale = b.gpu()
    for bad in ((q.float(), k, v, prefix, tables, lens), (q, k, v, prefix.long(), tables, lens),
                (q, k, v, prefix, tables[:1], lens), (q, k.bfloat16(), v, prefix, tables, lens),
                (q, k, v, prefix.cpu(), tables, lens)):
        with pytest.raises(ValueError):
            binding.decode_fp8_prefix(*bad, scale, b.ks, VS)


@pytest.mark.parametrize("D, S", [(64, 5), (128, 70)])
def test_every_code(D, S):
    """All finite codes in K and V, subnormal ones among them, and pools of subnormal codes alone."""
    for codes in (np.setdiff1d(np.arange(256), (0x7F, 0xFF)), np.r_[0:8, 0x80:0x88]):
        b = Batch(20, [3 + s % 40 for s in range(S)], 1, 8, 2, D, seed=7)
        rng = np.random.default_rng(9)
        for x in (b.k, b.v):
            real = x.numpy() != 0x7F
            x.numpy()[real] = rng.choice(codes, int(real.sum()))
        b.ks, b.scale = (0.0005, 0.1) if len(codes) > 16 else (2.0, 1.0)
        b.check("codes")


def test_nan_codes_stay_nan():
    """A NaN in a token that is seen reaches the rows that see it: a V entry its dimension, a K row all of them."""
    for D in (64, 128):
        b = Batch(20, [3, 50, -300], 1, 8, 2, D)
        out = b.check("clean")
        b.v[int(b.prefix[13]), 5, 1, 9] = 0x7F
        got = b.call(b.gpu())
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[:2, 4:, 9] = True
        assert torch.equal(torch.isnan(got), hit) and torch.equal(got[~hit], out[~hit])
        b.k[int(b.prefix[2]), 0, 0, 3] = 0xFF
        got = b.call(b.gpu())
        assert torch.isnan(got[:2, :4]).all() and not torch.isnan(got[2]).any()


def test_calls_on_two_streams_at_once():
    """Calls of both pool types overlap, each stream with scratch of its own."""
    b, plain = Batch(40, np.arange(60) % 30 + 1, 1, 8, 2, 128), bf16.Batch(30, [5, 60], 4, 16, 2, 64)
    args, other = b.gpu(), plain.gpu()
    want, want_plain = b.call(args), binding.decode_prefix(*other)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [(b.call(args, stream=streams[i % 2]), binding.decode_prefix(*other, stream=streams[1 - i % 2]))
           for i in range(12)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want) and torch.equal(y, want_plain)
