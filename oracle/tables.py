"""Plain restatement of one step's block tables and slot map (pa_tables_step),
one sequence after another on the host."""

from __future__ import annotations

import numpy as np

RELEASE = -1
ERR_BLOCK_ID, ERR_CONTEXT_LEN, ERR_SLOT, ERR_NO_BLOCKS = 1, 2, 4, 16


def tables_step(block_tables, context_lens, new_lens, free_blocks, free_count, block_size, max_tokens, prefix=()):
    """Returns (block_tables, context_lens, seq_starts, slot_mapping, free_blocks, free_count, error bits) after
    the step; the arguments are left as they are."""
    tables, stack = np.array(block_tables), np.array(free_blocks)
    lens = [int(c) for c in context_lens]
    width, bs, np_ = tables.shape[1], block_size, len(prefix)
    err = 0
    if not 0 <= free_count <= len(stack):
        err |= ERR_BLOCK_ID
        free_count = min(max(int(free_count), 0), len(stack))
    top = int(free_count)
    sound = [0 <= c <= width * bs and not 0 < c < np_ * bs and n >= RELEASE for c, n in zip(lens, new_lens)]
    if not all(sound):
        err |= ERR_CONTEXT_LEN
    for s, n in enumerate(new_lens):
        if sound[s] and n == RELEASE:
            for j in range(np_, -(-lens[s] // bs)):
                if top == len(stack):
                    err |= ERR_BLOCK_ID
                    break
                stack[top] = tables[s, j]
                top += 1
            lens[s] = 0
    slots, starts, stopped = [], [0], False
    # Blocks and tokens asked for so far, served or not: once they do not fit, nobody later is served.
    asked_blocks = asked_tokens = 0
    capacity = top
    for s, n in enumerate(new_lens):
        n = int(n)
        if sound[s] and n > 0:
            base = lens[s] if lens[s] else np_ * bs
            first, end = -(-base // bs), -(-(base + n) // bs)
            if base + n > width * bs:
                err |= ERR_CONTEXT_LEN
            else:
                asked_blocks += end - first
                asked_tokens += n
                if asked_blocks > capacity or asked_tokens > max_tokens:
                    err |= ERR_SLOT if asked_tokens > max_tokens else ERR_NO_BLOCKS
                else:
                    if lens[s] == 0:
                        tables[s, :np_] = prefix
                    for j in range(first, end):
                        top -= 1
                        tables[s, j] = stack[top]
                    slots += [int(tables[s, p // bs]) * bs + p % bs for p in range(base, base + n)]
                    lens[s] = base + n
        starts.append(len(slots))
    slots += [-1] * (max_tokens - len(slots))
    return (tables, np.array(lens, dtype=np.int32), np.array(starts, dtype=np.int32),
            np.array(slots, dtype=np.int64), stack, top, err)
