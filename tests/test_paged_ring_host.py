"""A model of the operand ring of the paged kernel of many rows: two groups of
fillers (keys, values) and one user, which see of a slot's barriers only the
parity of the last completed phase.  Whatever the order in which they get to
run, no slot is overwritten or read early, and none waits for ever."""
import random

import pytest


def plan(on, wide, lead, tiles, base, before):
    """Positions of key tile j (its first slot) and value tile j of a segment,
    as RingPlan has them."""
    def value(j):
        if on:
            return 2 * wide + (before + j) * (wide + 1)
        return base + min(lead, tiles) * wide + j + wide * min(j, max(tiles - lead, 0))

    def key(j):
        if on:
            return (before + j) * wide if before + j < 2 else value(j - 2) + 1
        return base + j * wide if j < lead else value(j - lead) + 1
    return key, value


def programs(wide, on, segments):
    keys, values, user = [], [], []
    base = before = 0
    for turns, tiles in segments:
        key, value = plan(on, wide, 2 if turns else 1, tiles, base, before)
        for j in range(tiles):
            keys += [key(j) + k for k in range(wide)]
            values.append(value(j))

        def logits(j):
            return [("use", key(j) + k) for k in range(wide)]

        def free(j):
            return [("free", key(j) + k) for k in range(wide)]
        if turns:
            for j in range(min(2, tiles)):
                user += logits(j) + free(j)
            for j in range(tiles):
                user += [("use", value(j)), ("free", value(j))]
                if j + 2 < tiles:
                    user += logits(j + 2) + free(j + 2)
        else:
            user += logits(0) + free(0)
            for j in range(tiles):
                user.append(("use", value(j)))
                user += logits(j + 1) if j + 1 < tiles else []
                user.append(("free", value(j)))
                user += free(j + 1) if j + 1 < tiles else []
        base += tiles * (wide + 1)
        before += tiles
    return keys, values, user


def run(slots, wide, on, segments, rng):
    progs = programs(wide, on, segments)
    full, empty, held, at = [0] * slots, [0] * slots, [None] * slots, [0, 0, 0]

    def passed(phases, n):  # a wait for the parity of phase n, with `phases` completed
        return n < 0 or (phases - 1) % 2 == n % 2

    while any(a < len(p) for a, p in zip(at, progs)):
        ready = []
        for who in (0, 1):
            if at[who] < len(progs[who]):
                pos = progs[who][at[who]]
                if passed(empty[pos % slots], pos // slots - 1):
                    ready.append(who)
        if at[2] < len(progs[2]):
            what, pos = progs[2][at[2]]
            if what == "free" or passed(full[pos % slots], pos // slots):
                ready.append(2)
        if not ready:
            return "nobody can go on"
        who = rng.choice(ready)
        if who < 2:
            pos = progs[who][at[who]]
            if held[pos % slots] is not None:
                return f"position {pos} written over {held[pos % slots]}"
            held[pos % slots] = pos
            full[pos % slots] += 1
        else:
            what, pos = progs[2][at[2]]
            if held[pos % slots] != pos:
                return f"{what} of {pos} finds {held[pos % slots]}"
            if what == "free":
                held[pos % slots] = None
                empty[pos % slots] += 1
        at[who] += 1
    return None


# (slots, slots of a key tile, order that runs on, kinds of segments)
VARIANTS = [(4, 1, False, (False, True)), (8, 1, False, (False, True)), (8, 2, False, (False, True)),
            (4, 2, True, (True,))]


@pytest.mark.parametrize("slots,wide,on,kinds", VARIANTS)
def test_ring_is_sound(slots, wide, on, kinds):
    rng = random.Random(slots * 10 + wide)
    for _ in range(1500):
        segments = [(rng.choice(kinds), rng.choice((1, 1, 2, 3, 4, 5, 9))) for _ in range(rng.randint(1, 8))]
        assert run(slots, wide, on, segments, rng) is None, segments


def test_model_sees_the_fault():
    """Four slots with two to a key tile and an order that starts anew with each
    segment: value tiles five positions apart take one phase for another."""
    rng = random.Random(1)
    found = [run(4, 2, False, [(True, rng.randint(1, 5)) for _ in range(6)], rng) for _ in range(200)]
    assert any(found)
