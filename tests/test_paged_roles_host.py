"""A model of the barriers of the paged kernel of many rows: fillers of keys and
of values, the issuing thread, the tensor pipe (which works off products and
commits in order), and two softmax warpgroups, of which each sees only the
parity of a barrier's last completed phase.  Whatever the order in which they
get to run, nobody waits for ever, and nothing is read before it was written or
overwritten before it was read."""
import random

import pytest

from tests.test_paged_ring_host import plan

NORMS = 8  # tiles whose scales are kept


class Stop(Exception):
    pass


class Bar:
    def __init__(self):
        self.phases = 0

    def passed(self, n):  # a wait for the parity of phase n
        return n < 0 or (self.phases - 1) % 2 == n % 2


class Model:
    """guard: q_full is used where a warpgroup has tiles alone; apart: the output
    has a barrier of its own (o_full)."""

    def __init__(self, slots, wide, on, segments, guard=True, apart=True):
        self.slots, self.wide, self.on, self.segments = slots, wide, on, segments
        self.guard, self.apart = guard, apart
        names = ["merge", "merged"] + [f"{n}{i}" for n in ("q", "s", "ph", "pf", "o") for i in (0, 1)]
        self.bar = {n: Bar() for n in names}
        self.full, self.empty = [Bar() for _ in range(slots)], [Bar() for _ in range(slots)]
        self.slot = [None] * slots
        self.scale = [None] * NORMS
        self.queries, self.logits, self.weights, self.out, self.ml = [None] * 2, [None] * 2, [None] * 2, [None] * 2, None
        self.pipe = []

    def need(self, what, found, wanted):
        if found != wanted:
            raise Stop(f"{what}: {found} instead of {wanted}")

    def each(self):
        base = before = 0
        for n, (turns, cnt) in enumerate(self.segments):
            tiles = max(cnt) if not turns else sum(cnt)
            key, value = plan(self.on, self.wide, 2 if turns else 1, tiles, base, before)
            yield n, turns, cnt, tiles, key, value, before
            base += tiles * (self.wide + 1)
            before += tiles

    # Roles: generators that yield a wait as (barrier, phase)
    def keys(self):
        for n, _, _, tiles, key, _, before in self.each():
            for j in range(tiles):
                for w in range(self.wide):
                    at = key(j) + w
                    yield self.empty[at % self.slots], at // self.slots - 1
                    self.need("slot", self.slot[at % self.slots], None)
                    self.slot[at % self.slots] = ("k", n, j, w)
                    if w == 0:
                        self.scale[(before + j) % NORMS] = (n, j)
                    self.full[at % self.slots].phases += 1

    def values(self):
        for n, _, _, tiles, _, value, _ in self.each():
            for j in range(tiles):
                at = value(j)
                yield self.empty[at % self.slots], at // self.slots - 1
                self.need("slot", self.slot[at % self.slots], None)
                self.slot[at % self.slots] = ("v", n, j, 0)
                self.full[at % self.slots].phases += 1

    def tensor(self):
        while True:
            while not self.pipe:
                yield None
            self.pipe.pop(0)()
            yield True

    def issue(self):
        used = {n: 0 for n in self.bar}

        def wait(name):
            used[name] += 1
            return self.bar[name], used[name] - 1

        def commit(bar):
            self.pipe.append(lambda: setattr(bar, "phases", bar.phases + 1))

        def free(pos, tag):
            def done():
                self.need("freed slot", self.slot[pos % self.slots], tag)
                self.slot[pos % self.slots] = None
                self.empty[pos % self.slots].phases += 1
            self.pipe.append(done)

        for n, turns, cnt, tiles, key, value, _ in self.each():
            def logits(i, j):
                for w in range(self.wide):
                    at = key(j) + w
                    yield self.full[at % self.slots], at // self.slots

                    def run(n=n, turns=turns, at=at, w=w):
                        self.need("key operand", self.slot[at % self.slots], ("k", n, j, w))
                        self.need("queries", self.queries[0 if turns else i], n)
                        self.logits[i] = (n, j)
                    self.pipe.append(run)
                commit(self.bar[f"s{i}"])

            def free_keys(j):
                for w in range(self.wide):
                    free(key(j) + w, ("k", n, j, w))

            def output(i, j, fresh, last):
                yield self.bar[f"ph{i}"], used[f"ph{i}"]
                used[f"ph{i}"] += 1
                yield self.full[value(j) % self.slots], value(j) // self.slots

                def half(n=n, value=value):
                    self.need("weights", self.weights[i][:3], (n, j, 0))
                    self.need("value operand", self.slot[value(j) % self.slots], ("v", n, j, 0))
                    if fresh:
                        self.need("output taken", self.out[i], None)
                self.pipe.append(half)
                yield wait(f"pf{i}")

                def rest(n=n):
                    self.need("weights", self.weights[i], (n, j, 0, 1))
                    self.out[i] = (n, last)
                self.pipe.append(rest)

            finished = (lambda i: commit(self.bar[f"o{i}"] if self.apart else self.bar[f"s{i}"]))
            for i in range(1 if turns else 2):
                if cnt[i] or not self.guard:
                    yield wait(f"q{i}")
            if turns:
                for j in range(min(2, tiles)):
                    yield from logits(j, j)
                    free_keys(j)
                for j in range(tiles):
                    yield from output(j & 1, j, j < 2, j + 2 >= tiles)
                    free(value(j), ("v", n, j, 0))
                    if j + 2 < tiles:
                        yield from logits(j & 1, j + 2)
                        free_keys(j + 2)
                    else:
                        finished(j & 1)
            else:
                for i in range(2):
                    if cnt[i]:
                        yield from logits(i, 0)
                free_keys(0)
                for j in range(tiles):
                    for i in range(2):
                        if j >= cnt[i]:
                            continue
                        yield from output(i, j, j == 0, j + 1 == cnt[i])
                        if j + 1 < cnt[i]:
                            yield from logits(i, j + 1)
                        else:
                            finished(i)
                    free(value(j), ("v", n, j, 0))
                    if j + 1 < tiles:
                        free_keys(j + 1)

    def softmax(self, i):
        ns = no = nm = 0
        for n, turns, cnt, _, _, _, before in self.each():
            if (cnt[i] or not self.guard) and (i == 0 or not turns):
                self.queries[i] = n
                yield True
                self.bar[f"q{i}"].phases += 1
            for m in range(cnt[i]):
                j = 2 * m + i if turns else m
                yield self.bar[f"s{i}"], ns
                ns += 1
                self.need("logits", self.logits[i], (n, j))
                self.need("scale", self.scale[(before + j) % NORMS], (n, j))
                self.weights[i] = (n, j, 0)
                yield True
                self.bar[f"ph{i}"].phases += 1
                yield True
                self.need("scale", self.scale[(before + j) % NORMS], (n, j))
                self.weights[i] = (n, j, 0, 1)
                yield True
                self.bar[f"pf{i}"].phases += 1
            if cnt[i]:
                if self.apart:
                    yield self.bar[f"o{i}"], no
                    no += 1
                else:
                    yield self.bar[f"s{i}"], ns
                    ns += 1
            if turns:
                if i == 1:
                    self.ml = n
                    yield True
                    self.bar["merge"].phases += 1
                    yield self.bar["merged"], nm
                else:
                    yield self.bar["merge"], nm
                    self.need("second result", self.ml, n)
                    for k in (0, 1):
                        if cnt[k]:
                            self.need("output", self.out[k], (n, True))
                            self.out[k] = None
                    yield True
                    self.bar["merged"].phases += 1
                nm += 1
            elif cnt[i]:
                self.need("output", self.out[i], (n, True))
                self.out[i] = None
                yield True

    def run(self, rng):
        roles = [self.keys(), self.values(), self.issue(), self.softmax(0), self.softmax(1), self.tensor()]
        waits = [next(r, "end") for r in roles]
        # how eager each role is: far apart, so that one may fall far behind
        weight = [rng.choice((1, 8, 64, 512)) for _ in roles]
        try:
            while any(w != "end" for w in waits[:5]):
                ready = [k for k, w in enumerate(waits) if w is True or (isinstance(w, tuple) and w[0].passed(w[1]))
                         or (w is None and self.pipe)]
                if not ready:
                    return "nobody can go on"
                k = rng.choices(ready, [weight[r] for r in ready])[0]
                waits[k] = next(roles[k], "end")
        except Stop as e:
            return str(e)
        return None


# slots, slots of a key tile, order that runs on, whether blocks of two query tiles occur
VARIANTS = [(4, 1, False, True), (8, 1, False, True), (8, 2, False, True), (4, 2, True, False),
            (4, 1, False, False), (6, 2, False, True), (3, 2, True, False)]  # the last three: fp16


def segments(rng, tall, first_unseen):
    out = []
    for _ in range(rng.randint(1, 7)):
        tiles = rng.choice((1, 1, 2, 3, 4, 5, 9))
        if not tall or rng.random() < 0.4:
            out.append((True, ((tiles + 1) // 2, tiles // 2)))
        else:  # the block's first 128 rows may see fewer of the run's tiles than its last, or none
            out.append((False, (rng.randint(0 if first_unseen else 1, tiles), tiles)))
    return out


@pytest.mark.parametrize("slots,wide,on,tall", VARIANTS)
def test_roles_are_sound(slots, wide, on, tall):
    rng = random.Random(slots * 10 + wide)
    for _ in range(700):
        s = segments(rng, tall, True)
        assert Model(slots, wide, on, s).run(rng) is None, s


def test_blocks_whose_first_rows_see_nothing():
    """Sequences with fewer keys than new tokens, as a batch padded in front has
    them: every segment's first 128 rows have no tile."""
    rng = random.Random(3)
    for n in (1, 2, 3, 4, 7):
        for _ in range(100):
            assert Model(4, 1, False, [(False, (0, 1))] * n).run(rng) is None
            assert Model(8, 1, False, [(False, (0, rng.randint(1, 3))) for _ in range(n)]).run(rng) is None


def test_model_sees_the_queries_fault():
    """A warpgroup without tiles that arrives on its queries' barrier all the same
    completes phases that the issuing thread never saw."""
    rng = random.Random(4)
    found = [Model(4, 1, False, [(False, (0, 1))] * 4, guard=False).run(rng) for _ in range(50)]
    assert any(f == "nobody can go on" for f in found)


def test_model_sees_the_outputs_fault():
    """One barrier for logits and output: behind a block of two query tiles, the
    logits of the next segment may complete it before the second warpgroup has
    seen that its output is there."""
    rng = random.Random(5)
    found = [Model(4, 1, False, [(False, (1, 1)), (True, (1, 1)), (False, (2, 2))], apart=False).run(rng)
             for _ in range(300)]
    assert any(found)
