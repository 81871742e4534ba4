"""A model of the decode kernel's producers, consumers and barriers under random
interleavings: waits go by the parity of a barrier's phase, as on the hardware.
With one producer filling every query slot no wait passes early and none is
missed; with the owner of a sequence's first tile filling it, a producer that
skipped sequences of few tiles passes early."""

import random

import pytest


def run(filler, tiles, stages, slots, rng, speed, producers=2, limit=20000):
    """None, or what went wrong.  Counters hold the completed phases of a barrier."""
    walk = [(s, j == 0) for s, n in enumerate(tiles) for j in range(n)]
    slot_free, slot_full = [0] * slots, [0] * slots
    stage_free, stage_full = [0] * stages, [0] * stages
    at, begun, done = [0] * producers, [False] * producers, 0

    def passes(completed, wanted):
        """(the wait returns, rightly): phases 0 .. wanted - 1 have to be complete."""
        return (completed ^ wanted) & 1 == 0, completed >= wanted

    for _ in range(limit):
        who = rng.choices(range(-1, producers), [speed] + [1] * producers)[0]
        if who < 0:  # the consumers, one tile
            s, first = walk[done]
            if stage_full[done % stages] <= done // stages:
                continue
            if first:
                if slot_full[s % slots] <= s // slots:
                    continue
                slot_free[s % slots] += 1
            stage_free[done % stages] += 1
            done += 1
            if done == len(walk):
                return None
            continue
        x = at[who]
        if x == len(walk):
            continue
        s, first = walk[x]
        mine = x % producers == who
        if first and not begun[who]:
            if filler(mine, who):
                ok, right = passes(slot_free[s % slots], s // slots)
                if not ok:
                    continue
                if not right:
                    return "a query slot filled early"
                slot_full[s % slots] += 1
            begun[who] = True
        if mine:
            ok, right = passes(stage_free[x % stages], x // stages)
            if not ok:
                continue
            if not right:
                return "a stage filled early"
            stage_full[x % stages] += 1
        at[who], begun[who] = x + 1, False
    return "stuck"


@pytest.mark.parametrize("stages", [2, 3, 4, 5, 6])
@pytest.mark.parametrize("slots", [1, 2])
def test_one_producer_fills_all_query_slots(stages, slots):
    rng = random.Random(stages * 10 + slots)
    for _ in range(60):
        tiles = [rng.choice([1, 1, 2, 3]) for _ in range(40)]
        assert run(lambda mine, who: who == 0, tiles, stages, slots, rng, rng.choice([0.1, 0.3, 1, 5])) is None


def test_the_owner_of_the_first_tile_would_fill_early():
    rng = random.Random(1)
    results = {run(lambda mine, who: mine, [rng.choice([1, 1, 2, 3]) for _ in range(40)], 6, 2, rng, 0.1, limit=5000)
               for _ in range(60)}
    assert "a query slot filled early" in results
