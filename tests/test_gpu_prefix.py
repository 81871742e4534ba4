"""GPU parity of decode over a shared prefix (pa_decode_prefix) against the fp64
restatement of multi-query decode.

Bound: the prefix's weights are rounded to bf16 (half a step, 2^-8) before they
meet V, scores and exponentials add less than 2^-13 to each weight, and the
output is rounded once."""

import numpy as np
import pytest
import torch

from oracle import modified
from paged_kv_cache_292_gb300 import binding

from paritylib import assert_rounded, captured, refused_under_capture

pytestmark = pytest.mark.gpu

WEIGHT_ERROR = 2.0**-8 + 2.0**-13


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


class Batch:
    """Sequences of `own` tokens behind a shared prefix of `blocks` blocks (own < 0: context blocks * bs + own).

    Rows of the pool without a token are NaN; rows of sharing sequences hold -1 for the prefix's blocks, which
    must not be read; `spread` scales the scores."""

    def __init__(self, blocks, own, Q=1, heads=8, kv_heads=2, D=128, bs=16, seed=0, spread=1.0, scale=None):
        rng = np.random.default_rng([seed, 5])
        own = np.asarray(own)
        S, P = len(own), blocks * bs
        self.ctx = np.where(own == -10**9, 0, P + own)
        self.S, self.Q, self.bs, self.D = S, Q, bs, D
        self.shares = self.ctx >= P + Q - 1
        nblk = -(-self.ctx // bs)
        width = int(max(nblk.max(), blocks)) + 2
        total = blocks + int(nblk.sum()) + 3
        order = rng.permutation(total)
        self.prefix = order[:blocks].astype(np.int32)
        full = np.full((S, width), -1, dtype=np.int32)
        at = blocks
        for s in range(S):
            skip = blocks if self.shares[s] else 0
            full[s, :skip] = self.prefix[:skip]
            n = int(nblk[s]) - skip
            full[s, skip : skip + n] = order[at : at + n]
            at += n
        self.full = full
        self.tables = full.copy()
        self.tables[self.shares, :blocks] = -1
        shape = (total, bs, kv_heads, D)
        self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        self.v = self.k.clone()
        for s in range(S):
            for t in range(int(self.ctx[s])):
                b, o = int(full[s, t // bs]), t % bs
                if t < P and self.shares[s] and s != int(np.argmax(self.shares)):
                    continue
                self.k[b, o] = torch.from_numpy(rng.standard_normal((kv_heads, D), dtype=np.float32) * spread)
                self.v[b, o] = torch.from_numpy(rng.standard_normal((kv_heads, D), dtype=np.float32))
        if not self.shares.any():  # a prefix that nobody has reached still lies in the pool
            for b in self.prefix:
                self.k[int(b)] = 1.0
                self.v[int(b)] = 2.0
        self.q = torch.from_numpy(rng.standard_normal((S, Q, heads, D), dtype=np.float32)).to(torch.bfloat16)
        self.scale = D**-0.5 if scale is None else scale

    def want(self):
        return modified.decode_mod(self.q.double().numpy(), np.nan_to_num(self.k.double().numpy()),
                                   np.nan_to_num(self.v.double().numpy()), self.full, self.ctx, self.scale, self.bs)

    def gpu(self):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
        q = self.q.cuda() if self.Q > 1 else self.q[:, 0].contiguous().cuda()
        return (q, self.k.cuda(), self.v.cuda(), i32(self.prefix), i32(self.tables), i32(self.ctx), self.scale)

    def check(self, what, **kw):
        args = self.gpu()
        out = torch.full_like(args[0], float("nan"))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        binding.decode_prefix(*args, out=out, error_flag=err, check_block_ids=True, **kw)
        torch.cuda.synchronize()
        assert int(err) == 0
        want, spread = self.want()
        assert_rounded(out.view(want.shape), want, spread, WEIGHT_ERROR, what)
        return out, args


NONE = -10**9  # an empty row


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads, kv_heads, Q", [(8, 2, 1), (3, 3, 1), (14, 2, 1), (8, 1, 1), (8, 2, 3), (16, 2, 4),
                                                 (5, 1, 6), (4, 4, 2)])
@pytest.mark.parametrize("blocks", [1, 8, 20])
def test_heads_and_queries(D, heads, kv_heads, Q, blocks):
    own = [Q, Q + 1, 40, 7 + Q, 130]
    Batch(blocks, own, Q, heads, kv_heads, D).check("heads")


@pytest.mark.parametrize("bs", [8, 16, 24, 32, 40, 64, 128, 256])
@pytest.mark.parametrize("tokens", [8, 120, 128, 136, 500, 1100])
def test_block_and_prefix_sizes(bs, tokens):
    Batch(max(1, tokens // bs), [1, 30, 2, 65], 1, 8, 2, 64, bs).check(f"bs={bs}")


@pytest.mark.parametrize("S", [1, 2, 31, 32, 33, 63, 64, 65, 97, 128, 130])
def test_numbers_of_rows(S):
    """Rows per KV head around one, two and three tiles of 128 (group 4)."""
    own = (np.arange(S) * 7) % 23 + 1
    Batch(9, own, 1, 8, 2, 64, 16, seed=S).check(f"S={S}")


def test_many_rows_and_several_queries():
    own = np.arange(70) % 9 + 4
    Batch(11, own, 4, 16, 2, 128, 32).check("many")


@pytest.mark.parametrize("Q", [1, 4])
def test_sequences_that_do_not_reach_the_prefixs_end(Q):
    """Empty rows, contexts inside the prefix, contexts that end with it."""
    own = [NONE, 5, -3, 0, Q - 1, Q, -100, NONE, 40, Q - 2]
    out, _ = Batch(8, own, Q, 8, 2, 128).check("short")
    assert torch.all(out[0] == 0) and torch.all(out[7] == 0)


def test_nobody_shares():
    Batch(8, [-5, NONE, -127, -60], 1, 8, 2, 128).check("nobody")


def test_no_prefix():
    Batch(0, [5, 17, 1, 100], 1, 8, 2, 128).check("none")
    Batch(0, [5, 17, 3, 100], 3, 8, 2, 64).check("none")


@pytest.mark.parametrize("spread", [0.0, 0.05, 6.0, 40.0])
def test_flat_and_peaked_scores(spread):
    """The running maximum moves little, or by hundreds of powers of two between tiles."""
    Batch(40, [3, 50, 200], 1, 8, 2, 128, seed=3, spread=spread).check("spread")


def test_rising_scores():
    """Keys that grow along the prefix: the maximum moves in every tile."""
    b = Batch(64, [1, 20], 1, 8, 2, 64, seed=5)
    for j, blk in enumerate(b.prefix):
        b.k[int(blk)] *= 0.1 * (j + 1)
    b.check("rising")


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_scales(scale):
    Batch(20, [3, 50, 200], 1, 8, 2, 128, seed=4, scale=scale).check("scale")


def test_long_prefix_of_small_batch():
    Batch(1100, [3, 50], 1, 4, 1, 64, 8).check("long")


def test_equals_multi_query_decode():
    b = Batch(30, [4, 9, 77], 3, 8, 2, 128)
    args = b.gpu()
    full = torch.from_numpy(b.full).cuda()
    got = binding.decode_prefix(*args)
    plain = binding.decode_multi(args[0], args[1], args[2], full, args[5], b.scale)
    _, spread = b.want()
    assert_rounded(got, plain.double().cpu().numpy(), spread, WEIGHT_ERROR + 2.0**-8, "against decode_multi")


def test_bad_prefix_block_is_reported():
    b = Batch(30, [4, 9, 77], 1, 8, 2, 128)
    b.tables[:, :30] = b.full[:, :30]
    for bad in (-1, b.k.shape[0], 2**31 - 1):
        args = b.gpu()
        args[3][7] = bad
        args[4][:, 7] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        binding.decode_prefix(*args, error_flag=err, check_block_ids=True)
        assert int(err) == binding.PA_DEVERR_BLOCK_ID


def test_workspace_of_any_content_capture_and_streams():
    """A caller's scratch filled with ones, shared by two captured graphs of different shapes on one stream."""
    batches = [Batch(30, np.arange(50) % 7 + 1, 1, 8, 2, 128), Batch(9, [5, 6], 4, 16, 2, 64)]
    size = max(binding.pa_decode_prefix_workspace_size(b.S, b.Q, b.q.shape[2], b.k.shape[2], b.D) for b in batches)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    parts = [(b, b.gpu()) for b in batches]
    outs = [torch.full_like(args[0], float("nan")) for _, args in parts]
    graphs = []
    for (b, args), out in zip(parts, outs):
        graphs.append(captured(lambda: binding.decode_prefix(*args, out=out, workspace=ws)))
    # Scratch of the library's own does not go into a graph.
    assert refused_under_capture(lambda: binding.decode_prefix(*parts[0][1]), binding.PagedAttnError)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    eager = [binding.decode_prefix(*args, stream=side) for _, args in parts]
    torch.cuda.synchronize()
    for (b, _), out, e in zip(parts, outs, eager):
        want, spread = b.want()
        assert_rounded(out.view(want.shape), want, spread, WEIGHT_ERROR, "captured")
        assert torch.equal(out, e)
    with pytest.raises(binding.PagedAttnError) as e:
        binding.decode_prefix(*parts[0][1], workspace=ws[: size // 64 // 256 * 256])
    assert e.value.code == binding.PA_ERR_WORKSPACE


def test_python_layer_refuses_mismatched_arguments():
    q, k, v, prefix, tables, lens, scale = Batch(8, [5, 6], 1, 8, 2, 64).gpu()
    for bad in ((q.float(), k, v, prefix, tables, lens), (q, k, v, prefix.long(), tables, lens),
                (q, k, v, prefix, tables[:1], lens), (q, k, v, prefix, tables, lens.long()),
                (q, k.float(), v, prefix, tables, lens), (q, k, v, prefix.cpu(), tables, lens)):
        with pytest.raises(ValueError):
            binding.decode_prefix(*bad, scale)
