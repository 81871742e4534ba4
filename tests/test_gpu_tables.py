"""pa_tables_step on the GPU against its restatement: every output is equal."""

import numpy as np
import pytest
import torch

from oracle import tables as oracle_tables
from paged_kv_cache_292_gb300 import binding

from paritylib import captured

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _state(rng, S, bs, max_ctx, np_, width, spare):
    """Sequences with contexts up to max_ctx behind a prefix of np_ blocks (some empty), and a shuffled free list."""
    lens = rng.integers(0, max_ctx + 1, S)
    lens = np.where(lens > 0, lens + np_ * bs, 0).astype(np.int32)
    held = [max(0, -(-int(c) // bs) - np_) for c in lens]
    order = rng.permutation(np_ + sum(held) + spare).astype(np.int32)
    prefix, at = order[:np_], np_
    tables = np.full((S, width), -1, dtype=np.int32)
    for s, n in enumerate(held):
        if lens[s]:
            tables[s, :np_] = prefix
        tables[s, np_ : np_ + n] = order[at : at + n]
        at += n
    free = np.full(len(order), -7, dtype=np.int32)
    free[: len(order) - at] = order[at:]
    return tables, lens, free, len(order) - at, prefix


def _gpu(tables, lens, new, free, count, bs, tokens, prefix, **kw):
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    d = dict(tables=t(tables), free=t(free), slots=torch.full((tokens,), -99, dtype=torch.int64, device="cuda"),
             err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    out = binding.tables_step(d["tables"], t(lens), t(new), d["free"], t([count]), bs, d["slots"],
                              prefix_table=t(prefix) if len(prefix) else None, error_flag=d["err"], **kw)
    torch.cuda.synchronize()
    return d["tables"], out[0], out[2], d["slots"], d["free"], out[1], d["err"]


def _check(args, **kw):
    want = oracle_tables.tables_step(*args)
    got = _gpu(*args, **kw)
    for name, g, w in zip(("tables", "lens", "starts", "slots", "free", "count", "err"), got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    return want


@pytest.mark.parametrize("S", [1, 2, 31, 33, 511, 513, 4096, 12288])
@pytest.mark.parametrize("bs, np_", [(16, 0), (1, 3), (24, 5)])
def test_mixed_steps(S, bs, np_):
    rng = np.random.default_rng([S, bs, np_])
    max_ctx = 9 * bs if S > 600 else 40 * bs
    width = np_ + 60
    tables, lens, free, count, prefix = _state(rng, S, bs, max_ctx, np_, width, 3 * S + 200)
    new = rng.choice([-1, 0, 1, 1, 1, 2, bs, 2 * bs + 1], S)
    tokens = int(new[new > 0].sum()) + 37
    want = _check((tables, lens, new, free, count, bs, tokens, prefix))
    assert want[6] in (0, oracle_tables.ERR_NO_BLOCKS)


@pytest.mark.parametrize("new", [[5000], [0], [-1], [1]])
@pytest.mark.parametrize("ctx", [0, 1, 16, 4000])
def test_one_sequence(ctx, new):
    rng = np.random.default_rng(ctx)
    tables, lens, free, count, prefix = _state(rng, 1, 16, 0, 0, 640, 640)
    lens[0] = ctx
    n = -(-ctx // 16)
    tables[0, :n], count = free[count - n : count], count - n
    _check((tables, lens, np.array(new), free, count, 16, 6000, prefix))


@pytest.mark.parametrize("short", ["blocks", "tokens", "row", "nothing free"])
def test_what_does_not_fit_is_not_served(short):
    rng = np.random.default_rng(5)
    tables, lens, free, count, prefix = _state(rng, 40, 8, 100, 2, 30, 300)
    new = rng.integers(1, 40, 40)
    tokens = int(new.sum())
    if short == "blocks":
        count = 25
    elif short == "tokens":
        tokens //= 2
    elif short == "row":
        new[7] = 1000
        new[11] = 2**31 - 1
    else:
        count = 0
    want = _check((tables, lens, new, free, count, 8, tokens, prefix))
    assert want[6] == {"blocks": 16, "tokens": 4, "row": 2, "nothing free": 16}[short]


def test_bad_lengths_and_counts_are_reported():
    rng = np.random.default_rng(6)
    tables, lens, free, count, prefix = _state(rng, 20, 8, 100, 2, 30, 100)
    lens[3], lens[4], lens[5], lens[6] = -5, 30 * 8 + 1, 7, 2**31 - 1
    new = np.full(20, 2)
    new[8], new[9], new[3], new[5] = -2, -2**31, 4, -1
    want = _check((tables, lens, new, free, count, 8, 64, prefix))
    assert want[6] == oracle_tables.ERR_CONTEXT_LEN
    for bad in (-1, len(free) + 5):
        _check((tables, np.abs(lens) * 0, np.full(20, 1), free, bad, 8, 64, prefix))


def test_more_returned_than_the_pool_has():
    """A free list that says the released blocks are free already: nothing is written beyond it."""
    rng = np.random.default_rng(7)
    tables, lens, free, count, prefix = _state(rng, 12, 8, 200, 0, 30, 10)
    new = np.full(12, -1)
    new[5] = 3
    want = _check((tables, lens, new, free, len(free) - 4, 8, 64, prefix))
    assert want[6] == oracle_tables.ERR_BLOCK_ID


def test_no_token_slots():
    rng = np.random.default_rng(8)
    tables, lens, free, count, prefix = _state(rng, 5, 8, 50, 0, 30, 10)
    _check((tables, lens, np.array([-1, 0, 0, -1, 0]), free, count, 8, 0, prefix))


def test_many_prompt_tokens():
    rng = np.random.default_rng(9)
    tables, lens, free, count, prefix = _state(rng, 700, 16, 300, 4, 600, 40000)
    new = rng.integers(1, 900, 700)
    _check((tables, lens, new, free, count, 16, int(new.sum()) + 1000, prefix))


def test_repeated_on_the_same_inputs_and_on_another_stream():
    rng = np.random.default_rng(10)
    tables, lens, free, count, prefix = _state(rng, 100, 16, 300, 4, 64, 400)
    new = rng.choice([-1, 0, 1, 30], 100)
    args = (tables, lens, new, free, count, 16, 2000, prefix)
    want = _check(args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    d_tables, d_free, slots = t(tables), t(free), torch.zeros(2000, dtype=torch.int64, device="cuda")
    d_lens, d_new, d_count, d_prefix = t(lens), t(new), t([count]), t(prefix)
    torch.cuda.synchronize()
    for _ in range(3):
        out = binding.tables_step(d_tables, d_lens, d_new, d_free, d_count, 16, slots, prefix_table=d_prefix,
                                  stream=side)
    torch.cuda.synchronize()
    assert np.array_equal(d_tables.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[3])
    assert np.array_equal(out[0].cpu().numpy(), want[1]) and np.array_equal(d_free.cpu().numpy(), want[4])


def test_captured_steps_swap_two_buffers():
    """A graph of two steps (a -> b, b -> a) replayed: the lengths and the free list move on by two steps each."""
    rng = np.random.default_rng(11)
    tables, lens, free, count, prefix = _state(rng, 64, 16, 100, 1, 64, 2000)
    new = np.ones(64, dtype=np.int32)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    d_tables, d_free, d_new, d_prefix = t(tables), t(free), t(new), t(prefix)
    la, lb, ca, cb = t(lens), t(lens), t([count]), t([count])
    starts, slots = t(np.zeros(65)), torch.zeros(64, dtype=torch.int64, device="cuda")
    kw = dict(prefix_table=d_prefix, seq_starts=starts)

    def two_steps():
        binding.tables_step(d_tables, la, d_new, d_free, ca, 16, slots, context_lens_out=lb, free_count_out=cb, **kw)
        binding.tables_step(d_tables, lb, d_new, d_free, cb, 16, slots, context_lens_out=la, free_count_out=ca, **kw)

    graph = captured(two_steps)
    state = (tables, lens, free, count)
    for _ in range(3):
        graph.replay()
        for _ in range(2):
            r = oracle_tables.tables_step(state[0], state[1], new, state[2], state[3], 16, 64, prefix)
            state = (r[0], r[1], r[4], r[5])
    torch.cuda.synchronize()
    assert np.array_equal(d_tables.cpu().numpy(), state[0]) and np.array_equal(la.cpu().numpy(), state[1])
    assert int(ca) == state[3] and np.array_equal(slots.cpu().numpy(), r[3])


@pytest.mark.parametrize("offset, tokens", [(0, 5001), (1, 5001), (1, 8), (1, 1), (3, 4098)])
def test_slot_buffers_of_any_alignment_and_length(offset, tokens):
    """A buffer that starts between 16-byte boundaries and ends inside a thread's run; nothing beyond it is written."""
    rng = np.random.default_rng([12, offset, tokens])
    tables, lens, free, count, prefix = _state(rng, 90, 8, 100, 1, 60, 2000)
    new = rng.choice([-1, 0, 1, 3, 60], 90)
    want = oracle_tables.tables_step(tables, lens, new, free, count, 8, tokens, prefix)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    room = torch.full((offset + tokens + 3,), -99, dtype=torch.int64, device="cuda")
    binding.tables_step(t(tables), t(lens), t(new), t(free), t([count]), 8, room[offset : offset + tokens],
                        prefix_table=t(prefix))
    got = room.cpu().numpy()
    assert np.array_equal(got[offset : offset + tokens], want[3])
    assert np.all(got[:offset] == -99) and np.all(got[offset + tokens :] == -99)
