"""pa_tables_step on the CPU: its refusals, and its restatement against the
host block manager (the same blocks in the same order)."""

import numpy as np
import pytest

from oracle import tables as oracle_tables
from paged_kv_cache_292_gb300 import binding
from paged_kv_cache_292_gb300 import build as pa_build


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return binding.load()


def _args(**kw):
    a = dict(block_tables=0x10000, context_lens_out=0x20000, seq_starts=0x30000, slot_mapping=0x40000,
             free_blocks=0x50000, free_count_out=0x60000, context_lens=0x70000, new_lens=0x80000,
             free_count=0x90000, prefix_table=None, num_prefix_blocks=0, num_seqs=4, max_blocks_per_seq=8,
             block_size=16, num_physical_blocks=32, max_tokens=64, stream=0, error_flag=None)
    a.update(kw)
    return list(a.values())


INVALID, UNSUPPORTED = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw, code", [
    *[({name: None}, INVALID) for name in ("block_tables", "context_lens_out", "seq_starts", "slot_mapping",
                                           "free_blocks", "free_count_out", "context_lens", "new_lens",
                                           "free_count")],
    (dict(num_seqs=0), INVALID),
    (dict(num_seqs=12289), UNSUPPORTED),
    (dict(max_blocks_per_seq=0), INVALID),
    (dict(block_size=0), INVALID),
    (dict(block_size=4097), UNSUPPORTED),
    (dict(max_blocks_per_seq=1 << 27), INVALID),  # 2^31 tokens a row
    (dict(num_physical_blocks=0), INVALID),
    (dict(max_tokens=-1), INVALID),
    (dict(num_prefix_blocks=-1), INVALID),
    (dict(num_prefix_blocks=2), INVALID),  # no prefix table
    (dict(num_prefix_blocks=9, prefix_table=0xa0000), INVALID),  # longer than a row
    (dict(context_lens=0x70002), INVALID),
    (dict(slot_mapping=0x40004), INVALID),
    (dict(context_lens_out=0x70000), INVALID),  # the input's own buffer
    (dict(context_lens_out=0x70000 + 12), INVALID),  # its last entry
    (dict(free_count_out=0x90000), INVALID),
    (dict(prefix_table=0x10000, num_prefix_blocks=2), INVALID),  # a row of the tables
    (dict(seq_starts=0x40000 + 8), INVALID),  # two outputs
])
def test_rejects_bad_arguments_on_host(lib, kw, code):
    assert lib.pa_tables_step(*_args(**kw)) == code
    assert lib.pa_last_error().decode()


def test_python_layer_wants_cuda_tensors():
    import torch

    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.tables_step(t.view(1, 4), t[:1], t[:1], t, t[:1], 16, torch.zeros(4, dtype=torch.int64))


@pytest.mark.parametrize("seed", range(4))
def test_restatement_hands_out_the_host_managers_blocks(lib, seed):
    """Appends only: the host manager hands out 0, 1, 2, ...; so does a stack that holds them in reverse."""
    rng = np.random.default_rng(seed)
    S, bs, nb, mb = 9, 4, 60, 12
    bm = binding.BlockManager(nb, bs, S, mb)
    tables = np.full((S, mb), -1, dtype=np.int32)
    lens, stack, count = np.zeros(S, dtype=np.int32), np.arange(nb, dtype=np.int32)[::-1].copy(), nb
    for _ in range(5):
        new = rng.integers(0, 6, S)
        slots, copies = bm.append_batch(list(range(S)), new.tolist())
        assert not copies
        tables, lens, starts, got, stack, count, err = oracle_tables.tables_step(tables, lens, new, stack, count, bs,
                                                                                 40)
        assert err == 0 and count == bm.num_free_blocks()
        assert np.array_equal(got[: starts[-1]], slots.numpy()) and np.all(got[starts[-1]:] == -1)
        want_tables, want_lens = bm.export()
        assert np.array_equal(tables, want_tables.numpy()) and np.array_equal(lens, want_lens.numpy())


def test_restatement_by_hand():
    """Blocks of 4, prefix of one block (id 9): one sequence leaves, one starts, one grows into a new block."""
    tables = np.array([[9, 5, -1], [-1, -1, -1], [9, 6, -1]], dtype=np.int32)
    stack = np.array([1, 2, 0, 0, 0, 0, 0, 0, 0, 0], dtype=np.int32)
    t, lens, starts, slots, stack, count, err = oracle_tables.tables_step(
        tables, [7, 0, 8], [-1, 5, 1], stack, 2, 4, 8, prefix=(9,))
    # Sequence 0 returns block 5 (stack 1, 2, 5); sequence 1 holds the prefix and takes 5 and 2; sequence 2 takes 1.
    assert err == 0 and count == 0 and lens.tolist() == [0, 9, 9]
    assert t.tolist() == [[9, 5, -1], [9, 5, 2], [9, 6, 1]]
    assert starts.tolist() == [0, 0, 5, 6]
    assert slots.tolist() == [20, 21, 22, 23, 8, 4, -1, -1]
