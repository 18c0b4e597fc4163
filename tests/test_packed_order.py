"""The barriers of the packed attention's forward (csrc/kda_packed_fwd.cu), as a model without a GPU: one
CTA's loads, issuing thread, tensor pipe and softmax warps, stepped in any order. A barrier is what the
hardware has: a count of completed phases of which a wait sees the parity alone, so a wait for a phase is
over too early if the one before it is not complete, and never if the one behind it is.

Numbers of barriers, what completes them, and the order of the products are the kernel's; each role waits
for what the kernel's waits for. Copies land in any order. Items are known to every role beforehand, which
leaves the roles freer than the kernel's hand-out does."""
import itertools
import random

import pytest


class Stopped(Exception):
    """No role can go on."""


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.done = 0  # completed phases

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def over(self, phase):
        """try_wait.parity of phase number `phase`."""
        if self.done & 1 == phase & 1:
            return False
        assert self.done == phase + 1, "a wait ended before its phase"
        return True


class Model:
    """items: (key tiles of stream 0, of stream 1) of each. rescale: how often a warp rescales its outputs. places: tiles of scores in TMEM; three: heads of
    64, two: heads of 128 (one for each stream). barriers of scores and probabilities: "own", one for each
    stream and place, as the kernel has; "shared", one for each place; "parity", two for each stream, by the parity of its tile."""

    def __init__(self, items, places=3, barriers="own", warps=2, rescale=0.5):
        self.rescale, self.rng = rescale, random.Random(len(items))
        self.items, self.places, self.barriers, self.warps = items, places, barriers, warps
        self.slots = 6 if places == 3 else 5
        keys = {self.key(s, j, place) for s in range(2) for j in range(2) for place in range(3)}
        self.s_full = {i: Barrier(1) for i in keys}
        self.p_ready = {i: Barrier(warps) for i in keys}
        self.phases = {}  # of each tile's barriers
        used, tile = dict.fromkeys(keys, 0), [0, 0]
        for t in self.tiles():
            k = self.key(t[1], tile[t[1]], self.place(*t))
            tile[t[1]] += 1
            self.phases[t], used[k] = (k, used[k]), used[k] + 1
        self.full, self.empty = ([Barrier(1) for _ in range(self.slots)] for _ in range(2))
        self.q_full, self.q_empty = Barrier(1), Barrier(1)
        self.o_done, self.o_free = [Barrier(1) for _ in range(2)], [Barrier(warps) for _ in range(2)]
        self.pipe = []      # products and commits that were issued
        self.copies = []    # in flight: (what, where, barrier)
        self.ring, self.q = [None] * self.slots, None
        self.tmem, self.read = [None] * places, [0] * places  # what lies in a place; warps that have made P of it
        self.o, self.written = [None, None], []

    # ---- what is issued, and what runs when its turn comes ----
    def commit(self, bar):
        self.pipe.append(bar.arrive)

    def scores(self, item, s, j, place, slot):
        def run():
            assert self.ring[slot][:2] == (item, j) and self.q == item
            assert self.tmem[place] is None, "scores over others"
            self.tmem[place], self.read[place] = ("S", item, s, j), 0
        self.pipe.append(run)

    def outputs(self, item, s, j, place, slot):
        def run():
            assert self.ring[slot][:2] == (item, j) and self.tmem[place] == ("P", item, s, j)
            if j == 0:
                assert self.o[s] is None, "outputs over others"
            else:
                assert self.o[s] == (item, j - 1)
            self.tmem[place], self.o[s] = None, (item, j)
        self.pipe.append(run)

    def land(self, k):
        what, where, bar = self.copies.pop(k)
        if where is None:
            self.q = what
        else:
            self.ring[where] = what
        bar.arrive()

    def tiles(self):
        """All tiles of the call, (item, stream, tile of it), in the order of their products."""
        for i, n in enumerate(self.items):
            for j, s in sorted((j, s) for s in range(2) for j in range(n[s])):
                yield i, s, j

    def place(self, i, s, j):
        """Where a tile's scores lie: the streams' tiles take three places in turn, from the first in every item."""
        n = self.items[i]
        return s if self.places == 2 else (j if n[1] == 0 else 2 * j + (s if j < n[0] else 0)) % 3

    def key(self, s, tile, place):
        """A tile's barriers. tile: number among all of the stream's."""
        if self.places == 2:
            return s
        return {"own": (s, place), "shared": place, "parity": (s, tile % 2)}[self.barriers]

    # ---- roles: generators of what they wait for ----
    def load(self):
        k = 0
        for i, n in enumerate(self.items):
            if i > 0:
                yield lambda: self.q_empty.over(i - 1)
            self.copies.append((i, None, self.q_full))
            for j in range(max(n)):
                for v in range(1 if self.places == 3 else 2):  # K and V together, or in turn
                    slot, turn = k % self.slots, k // self.slots
                    if turn > 0:
                        yield lambda: self.empty[slot].over(turn - 1)
                    self.copies.append(((i, j, v), slot, self.full[slot]))
                    k += 1

    def issue3(self):
        used, pos0 = [0, 0], 0
        for i, n in enumerate(self.items):
            two, nk = n[1] > 0, max(n)
            mine = [t for t in self.tiles() if t[0] == i]

            def score(t):
                _, s, j = t
                self.scores(i, s, j, self.place(*t), (pos0 + j) % 6)
                self.commit(self.s_full[self.phases[t][0]])
                if s == two and j + 1 == nk:
                    self.commit(self.q_empty)

            def keys(t):
                return self.full[(pos0 + t[2]) % 6].over((pos0 + t[2]) // 6)

            for t in mine[:3]:
                yield lambda: self.q_full.over(i)
                yield lambda: keys(t)
                score(t)
            for g, t in enumerate(mine):
                _, s, j = t
                ahead = mine[g + 3] if g + 3 < len(mine) else None
                fresh = ahead and (ahead[1] == 0 or ahead[2] >= n[0])  # the first with its keys
                bar, phase = self.phases[t]
                yield lambda: self.p_ready[bar].over(phase) and (not fresh or keys(ahead))
                if j == 0:
                    used[s] += 1
                    if used[s] > 1:
                        yield lambda: self.o_free[s].over(used[s] - 2)
                self.outputs(i, s, j, self.place(*t), (pos0 + j) % 6)
                if ahead:
                    score(ahead)
                if s == two:
                    self.commit(self.empty[(pos0 + j) % 6])
                if j + 1 == n[s]:
                    self.commit(self.o_done[s])
            pos0 += nk

    def issue2(self):
        before, used, k = [0, 0], [0, 0], 0
        for i, n in enumerate(self.items):
            nk = max(n)
            yield lambda: self.q_full.over(i) and self.full[k % 5].over(k // 5)
            for s in range(2):
                if n[s]:
                    self.scores(i, s, 0, s, k % 5)
                    self.commit(self.s_full[s])
            self.commit(self.empty[k % 5])
            if nk == 1:
                self.commit(self.q_empty)
            for j in range(nk):
                v, k, more = k + 1, k + 2, j + 1 < nk
                for s in range(2):
                    if j >= n[s]:
                        continue
                    yield lambda: (self.p_ready[s].over(before[s] + j) and self.full[v % 5].over(v // 5)
                                   and (not more or self.full[k % 5].over(k // 5)))
                    if j == 0:
                        used[s] += 1
                        if used[s] > 1:
                            yield lambda: self.o_free[s].over(used[s] - 2)
                    self.outputs(i, s, j, s, v % 5)
                    if j + 1 == n[s]:
                        self.commit(self.o_done[s])
                    if j + 1 < n[s]:
                        self.scores(i, s, j + 1, s, k % 5)
                        self.commit(self.s_full[s])
                self.commit(self.empty[v % 5])
                if more:
                    self.commit(self.empty[k % 5])
                if j + 2 == nk:
                    self.commit(self.q_empty)
            before = [before[s] + n[s] for s in range(2)]

    def softmax(self, s):
        done, pos0 = 0, 0
        for i, n in enumerate(self.items):
            for j in range(n[s]):
                place, (bar, phase) = self.place(i, s, j), self.phases[i, s, j]
                yield lambda: self.s_full[bar].over(phase)
                assert self.tmem[place] == ("S", i, s, j)
                if j + 1 == n[s]:  # rows past the sequence are cleared in V
                    at = pos0 + (j if self.places == 3 else 2 * j + 1)
                    yield lambda: self.full[at % self.slots].over(at // self.slots)
                if j > 0 and self.rng.random() < self.rescale:
                    if self.places == 3:
                        at = pos0 + j - 1
                        yield lambda: self.empty[at % self.slots].over(at // self.slots)
                    assert self.o[s] == (i, j - 1)
                yield lambda: True  # arithmetic
                self.read[place] += 1
                if self.read[place] == self.warps:
                    self.tmem[place] = ("P", i, s, j)
                self.p_ready[bar].arrive()
            pos0 += max(n) * (1 if self.places == 3 else 2)
            if n[s] == 0:
                continue
            yield lambda: self.o_done[s].over(done)
            done += 1
            assert self.o[s] == (i, n[s] - 1)
            yield lambda: True  # outputs are written
            self.written.append((i, s))
            if self.written.count((i, s)) == self.warps:
                self.o[s] = None
            self.o_free[s].arrive()

    def run(self, choose):
        """choose(names of what can go on): the one that does."""
        roles = {"load": self.load(), "issue": self.issue3() if self.places == 3 else self.issue2()}
        for s in range(2):
            for w in range(self.warps):
                roles[f"softmax {s} {w}"] = self.softmax(s)
        waits = {r: (lambda: True) for r in roles}
        while roles or self.pipe or self.copies:
            can = [r for r in roles if waits[r]()]
            can += ["pipe"] * bool(self.pipe) + [f"copy {k}" for k in range(len(self.copies))]
            if not can:
                raise Stopped(sorted(roles))
            r = choose(can)
            if r == "pipe":
                self.pipe.pop(0)()
            elif r.startswith("copy"):
                self.land(int(r.split()[1]))
            else:
                waits[r] = next(roles[r], None)
                if waits[r] is None:
                    del roles[r]
        assert sorted(set(self.written)) == [(i, s) for i, n in enumerate(self.items) for s in range(2) if n[s]]


def last(names):
    """A role (or several) that goes on only where nothing else can."""
    def choose(can):
        others = [r for r in can if not r.startswith(names)]
        return (others or can)[0]
    return choose


def at_random(seed):
    rng = random.Random(seed)
    weight = {r: 4.0 ** rng.uniform(-3, 3) for r in ("load", "issue", "softmax 0", "softmax 1", "pipe", "copy")}
    def choose(can):
        return rng.choices(can, [next(w for k, w in weight.items() if r.startswith(k)) for r in can])[0]
    return choose


def orders(seeds):
    for names in ("softmax", "softmax 0", "softmax 1", "softmax 0 0", "softmax 1 1", "load", "copy", "issue", "pipe",
                  ("copy", "load"), ("softmax", "load"), ("softmax", "copy"), ("issue", "pipe")):
        yield last(names)
    for seed in range(seeds):
        yield at_random(seed)


SHAPES = [(1, 0), (1, 2), (3, 0), (3, 4), (5, 0)]  # (2 w - 1, 2 w), or without the second stream


@pytest.mark.parametrize("places", [3, 2])
def test_no_order_of_events_stops_the_forward(places):
    for items in itertools.product(SHAPES, repeat=3):
        for choose in orders(6):
            Model(items, places).run(choose)


@pytest.mark.parametrize("places", [3, 2])
def test_longer_runs_of_items(places):
    rng = random.Random(places)
    for seed in range(60):
        items = [rng.choice(SHAPES + [(7, 0), (7, 8), (9, 0)]) for _ in range(8)]
        Model(items, places, warps=4).run(at_random(seed))


def test_the_model_finds_barriers_that_complete_twice():
    """Two barriers a stream, by the parity of its tile, do not hold where one stream's scores are issued three
    tiles ahead: tiles 0 and 2 share one, and nothing holds the second back until the first is seen."""
    with pytest.raises(Stopped):
        Model([(3, 0), (3, 0)], barriers="parity").run(last("softmax"))  # scores: behind late warps
    with pytest.raises(Stopped):
        Model([(5, 0)], barriers="parity", rescale=0).run(last("copy"))  # probabilities: before late keys
    for choose in orders(20):  # items of two streams have two tiles of one ahead
        Model([(3, 4), (5, 6), (1, 2)], barriers="parity").run(choose)


def test_the_model_finds_waits_that_end_too_early():
    """One barrier a place for both streams: one that had no part in an item waits for a phase whose forerunner it
    has not seen."""
    with pytest.raises(AssertionError, match="before its phase"):
        Model([(3, 0), (3, 4)], barriers="shared").run(last("pipe"))
