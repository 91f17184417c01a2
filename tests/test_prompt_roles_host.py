"""A model of the barriers of the prompt kernel: the loading warp, copies that
complete in any order, the guard of the values, the issuing thread, the tensor
pipe (which works off products and commits in order) and two softmax
warpgroups, of which each sees only the parity of a barrier's last completed
phase.  Whatever the order in which they get to run, nobody waits for ever, and
nothing is read before it was written or overwritten before it was read."""
import random

from tests.test_paged_roles_host import Bar, Stop

STAGES = 2


class Model:
    """items: key tiles of the two query tiles.  apart: the output has a barrier
    of its own (o_full)."""

    def __init__(self, items, apart=True):
        self.items, self.apart = items, apart
        names = [f"{n}{i}" for n in ("qf", "qe", "kf", "ke", "vf", "vok", "ve", "s", "ph", "pf", "o", "if", "ie")
                 for i in (0, 1)]
        self.bar = {n: Bar() for n in names}
        self.mem = {f"{n}{i}": None for n in ("q", "k", "v", "s", "p", "o") for i in (0, 1)}
        self.item, self.taken = [None, None], [0, 0]
        self.copies, self.pipe = [], []

    def need(self, what, found, wanted):
        if found != wanted:
            raise Stop(f"{what}: {found} instead of {wanted}")

    def done(self, name):
        self.bar[name].phases += 1

    def take(self, k):
        yield self.bar[f"if{k & 1}"], k >> 1
        self.need("item", self.item[k & 1], k)
        self.taken[k & 1] += 1
        if self.taken[k & 1] == 4:
            self.taken[k & 1] = 0
            self.done(f"ie{k & 1}")

    def copy(self, place, what, bar):
        def run():
            self.mem[place] = what
            self.done(bar)
        self.copies.append(run)

    def load(self):
        keys = values = 0
        queries = [0, 0]
        for k in range(len(self.items) + 1):
            if k >= 2:
                yield self.bar[f"ie{k & 1}"], (k >> 1) - 1
            self.item[k & 1] = k
            self.done(f"if{k & 1}")
            yield True
            if k == len(self.items):
                return
            cnt = self.items[k]
            for j in range(max(cnt)):
                st = keys % STAGES
                yield self.bar[f"ke{st}"], keys // STAGES - 1
                self.copy(f"k{st}", (k, j), f"kf{st}")
                keys += 1
                for i in range(2):
                    if j == 0 and cnt[i]:
                        yield self.bar[f"qe{i}"], queries[i] - 1
                        self.copy(f"q{i}", k, f"qf{i}")
                        queries[i] += 1
                yield self.bar[f"ve{st}"], values // STAGES - 1
                self.copy(f"v{st}", (k, j), f"vf{st}")
                values += 1

    def guard(self):
        pos = 0
        for k, cnt in enumerate(self.items + [None]):
            yield from self.take(k)
            for j in range(max(cnt) if cnt else 0):
                yield self.bar[f"vf{pos % STAGES}"], pos // STAGES
                self.need("guarded values", self.mem[f"v{pos % STAGES}"], (k, j))
                yield True
                self.done(f"vok{pos % STAGES}")
                pos += 1

    def memory(self, rng):
        while True:
            while not self.copies:
                yield None
            self.copies.pop(rng.randrange(len(self.copies)))()
            yield True

    def tensor(self):
        while True:
            while not self.pipe:
                yield None
            self.pipe.pop(0)()
            yield True

    def issue(self):
        nq, np, pos = [0, 0], [0, 0], 0

        def commit(name):
            self.pipe.append(lambda: self.done(name))

        def logits(i, k, j, pos, last):
            def run():
                self.need("queries", self.mem[f"q{i}"], k)
                self.need("keys", self.mem[f"k{pos % STAGES}"], (k, j))
                self.mem[f"s{i}"] = (k, j)
            self.pipe.append(run)
            commit(f"s{i}")
            if last:
                commit(f"qe{i}")

        for k, cnt in enumerate(self.items + [None]):
            yield from self.take(k)
            if cnt is None:
                return
            yield self.bar[f"kf{pos % STAGES}"], pos // STAGES
            for i in range(2):
                if cnt[i]:
                    yield self.bar[f"qf{i}"], nq[i]
                    nq[i] += 1
                    logits(i, k, 0, pos, cnt[i] == 1)
            commit(f"ke{pos % STAGES}")
            for j in range(max(cnt)):
                have = False
                for i in range(2):
                    if j >= cnt[i]:
                        continue
                    yield self.bar[f"ph{i}"], np[i]
                    yield self.bar[f"vok{pos % STAGES}"], pos // STAGES

                    def half(i=i, k=k, j=j, pos=pos):
                        self.need("weights", self.mem[f"p{i}"][:3], (k, j, 0))
                        self.need("values", self.mem[f"v{pos % STAGES}"], (k, j))
                        if j == 0:
                            self.need("output taken", self.mem[f"o{i}"], None)
                    self.pipe.append(half)
                    yield self.bar[f"pf{i}"], np[i]
                    np[i] += 1

                    def rest(i=i, k=k, j=j, last=j + 1 == cnt[i]):
                        self.need("weights", self.mem[f"p{i}"], (k, j, 0, 1))
                        self.mem[f"o{i}"] = (k, last)
                    self.pipe.append(rest)
                    if j + 1 < cnt[i]:
                        if not have:
                            yield self.bar[f"kf{(pos + 1) % STAGES}"], (pos + 1) // STAGES
                        have = True
                        logits(i, k, j + 1, pos + 1, j + 2 == cnt[i])
                    else:
                        commit(f"o{i}" if self.apart else f"s{i}")
                commit(f"ve{pos % STAGES}")
                if j + 1 < max(cnt):
                    commit(f"ke{(pos + 1) % STAGES}")
                pos += 1

    def softmax(self, i):
        ns = no = 0
        for k, cnt in enumerate(self.items + [None]):
            yield from self.take(k)
            if cnt is None or not cnt[i]:
                continue
            for j in range(cnt[i]):
                yield self.bar[f"s{i}"], ns
                ns += 1
                self.need("logits", self.mem[f"s{i}"], (k, j))
                self.mem[f"p{i}"] = (k, j, 0)
                yield True
                self.done(f"ph{i}")
                self.mem[f"p{i}"] = (k, j, 0, 1)
                yield True
                self.done(f"pf{i}")
            if self.apart:
                yield self.bar[f"o{i}"], no
                no += 1
            else:
                yield self.bar[f"s{i}"], ns
                ns += 1
            self.need("output", self.mem[f"o{i}"], (k, True))
            self.mem[f"o{i}"] = None
            yield True

    def run(self, rng):
        roles = [self.load(), self.guard(), self.issue(), self.softmax(0), self.softmax(1), self.memory(rng),
                 self.tensor()]
        queues = {5: self.copies, 6: self.pipe}
        try:
            waits = [next(r, "end") for r in roles]
            weight = [rng.choice((1, 8, 64, 512)) for _ in roles]
            while any(w != "end" for w in waits[:5]):
                ready = [n for n, w in enumerate(waits) if w is True or (w is None and queues[n])
                         or (isinstance(w, tuple) and w[0].passed(w[1]))]
                if not ready:
                    return "nobody can go on"
                n = rng.choices(ready, [weight[r] for r in ready])[0]
                waits[n] = next(roles[n], "end")
        except Stop as e:
            return str(e)
        return None


def items(rng):
    out = []
    for _ in range(rng.randint(1, 6)):
        a = rng.choice((1, 1, 2, 3, 5))
        out.append((a, rng.choice((0, a, a + 1))))  # the second tile may lie behind the end
    return out


def test_roles_are_sound():
    rng = random.Random(1)
    for _ in range(2500):
        s = items(rng)
        assert Model(s).run(rng) is None, s


def test_model_sees_the_outputs_fault():
    """One barrier for logits and output: the next item's logits may complete it
    before the softmax has seen that the output is there."""
    rng = random.Random(2)
    assert any(Model([(1, 1), (1, 1), (2, 0)], apart=False).run(rng) for _ in range(300))
