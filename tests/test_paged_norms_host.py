"""A model of how the four warps that expand a tile find its largest norm: each
puts its own down, all meet at a barrier, each reads the four.  Two places are
used alternately; no warp may overwrite one that another has still to read."""
import random

import pytest


def run(segments, run_on, rng):
    """Whether some warp reads a place that holds another tile's norm.  run_on: the
    places alternate over the whole run, not anew in each segment."""
    places = [[None] * 4, [None] * 4]
    tiles = [(n, j) for n, count in enumerate(segments) for j in range(count)]
    met = [0] * len(tiles)
    turn = [i if run_on else j for i, (_, j) in enumerate(tiles)]

    def warp(w):
        for i, tile in enumerate(tiles):
            places[turn[i] & 1][w] = tile
            met[i] += 1
            while met[i] < 4:
                yield True
            for other in range(4):  # (read one after the other)
                if places[turn[i] & 1][other] != tile:
                    yield False
                yield True

    warps = [warp(w) for w in range(4)]
    weight = [rng.choice((1, 8, 64)) for _ in warps]
    left = list(range(4))
    while left:
        w = rng.choices(left, [weight[x] for x in left])[0]
        step = next(warps[w], None)
        if step is False:
            return True
        if step is None:
            left.remove(w)
    return False


@pytest.mark.parametrize("most", [1, 2, 3, 9])
def test_places_alternate_over_the_run(most):
    rng = random.Random(most)
    for _ in range(400):
        assert not run([rng.randint(1, most) for _ in range(rng.randint(1, 6))], True, rng)


def test_model_sees_the_fault():
    """Segments of an odd number of tiles, places counted anew in each."""
    rng = random.Random(7)
    assert any(run([1, 3, 1, 1], False, rng) for _ in range(100))
    assert not any(run([2, 4, 2], False, rng) for _ in range(100))
