"""The barriers of the packed attention's kernels (csrc/kda_packed_fwd.cu, kda_packed_bwd.cu), as models without a
GPU: one CTA's loads, issuing thread, tensor pipe and warps of arithmetic, stepped in any order. A barrier is what the
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


class Steps:
    """What the models share: a pipe of products and commits in order, copies that land in any, and roles,
    generators of what they wait for."""

    def commit(self, bar):
        self.pipe.append(bar.arrive)

    def run(self, choose):
        """choose(names of what can go on): the one that does."""
        roles = dict(self.roles())
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
        assert self.finished()


class Model(Steps):
    """The forward. items: (key tiles of stream 0, of stream 1) of each. rescale: how often a warp rescales its outputs. places: tiles of scores in TMEM; three: heads of
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

    def roles(self):
        yield "load", self.load()
        yield "issue", self.issue3() if self.places == 3 else self.issue2()
        for s in range(2):
            for w in range(self.warps):
                yield f"softmax {s} {w}", self.softmax(s)

    def finished(self):
        return sorted(set(self.written)) == [(i, s) for i, n in enumerate(self.items) for s in range(2) if n[s]]


def last(names):
    """A role (or several) that goes on only where nothing else can."""
    def choose(can):
        others = [r for r in can if not r.startswith(names)]
        return (others or can)[0]
    return choose


def at_random(seed):
    rng = random.Random(seed)
    weight = {r: 4.0 ** rng.uniform(-3, 3) for r in ("load", "issue", "softmax 0", "softmax 1", "math", "pipe", "copy")}
    def choose(can):
        return rng.choices(can, [next(w for k, w in weight.items() if r.startswith(k)) for r in can])[0]
    return choose


def orders(seeds):
    for names in ("math", "math 0", "load q", "softmax", "softmax 0", "softmax 1", "softmax 0 0", "softmax 1 1", "load", "copy", "issue", "pipe",
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


class Backward(Steps):
    """What the backward's passes share. Every warp of arithmetic takes part in every tile."""

    def __init__(self, items, warps=3):
        self.items, self.warps = items, warps
        self.pipe, self.copies, self.loaded = [], [], {}
        self.s_full, self.done, self.acc_free = Barrier(1), Barrier(1), Barrier(warps)
        self.acc, self.out = None, 0  # the accumulators' last step; items written, by each warp

    def copy(self, key, what, bar):
        """key: where; what: as the products name it."""
        self.copies.append((key, what, bar))

    def land(self, k):
        key, what, bar = self.copies.pop(k)
        self.loaded[key] = what
        bar.arrive()

    def finished(self):
        return self.out == self.warps * len(self.items)


class KeysAndValues(Backward):
    """dk, dv. items: steps of each; every third step's last rows are another sequence's."""

    def __init__(self, items, slots=(3, 2), warps=3):
        super().__init__(items, warps)
        self.q_full, self.q_empty = ([Barrier(1) for _ in range(slots[0])] for _ in range(2))
        self.do_full, self.do_empty = [Barrier(1) for _ in range(slots[1])], [Barrier(1 + warps) for _ in range(slots[1])]
        self.kv_full, self.kv_empty = Barrier(2), Barrier(1)
        self.dp_full, self.p_ready, self.ds_ready = Barrier(1), Barrier(warps), Barrier(warps)
        self.s = self.dp = None  # what lies there: ("S", step), or ("P", step) once every warp has written
        self.wrote = {}

    def roles(self):
        yield "load q", self.load(self.q_full, self.q_empty, "q", True)
        yield "load do", self.load(self.do_full, self.do_empty, "do", False)
        yield "issue", self.issue()
        for w in range(self.warps):
            yield f"math {w}", self.math()

    def load(self, full, empty, name, first):
        t = 0
        for i, steps in enumerate(self.items):
            if first:
                if i > 0:
                    yield lambda: self.kv_empty.over(i - 1)
                self.copy("k", i, self.kv_full)
                self.copy("v", i, self.kv_full)
            for _ in range(steps):
                slot, turn = t % len(full), t // len(full)
                if turn > 0:
                    yield lambda: empty[slot].over(turn - 1)
                self.copy((name, slot), t, full[slot])
                t += 1

    def issue(self):
        def product(check, **to):
            def run():
                assert check()
                vars(self).update(to)
            self.pipe.append(run)

        def full(bars, t):
            return bars[t % len(bars)].over(t // len(bars))

        def has(i, t, name):
            n = len(self.q_full if name == "q" else self.do_full)
            return self.loaded["k"] == i and self.loaded["v"] == i and self.loaded[name, t % n] == t

        def scores(i, t):
            product(lambda: has(i, t, "q") and self.s in (None, ("used",)), s=("S", t))
            self.commit(self.s_full)

        def dp(i, t):
            product(lambda: has(i, t, "do") and self.dp in (None, ("used",)), dp=("S", t))
            self.commit(self.dp_full)

        t = 0
        for i, steps in enumerate(self.items):
            yield lambda: self.kv_full.over(i) and full(self.q_full, t) and full(self.do_full, t)
            scores(i, t)
            dp(i, t)
            if steps == 1:
                self.commit(self.kv_empty)
            for n in range(steps):
                more = n + 1 < steps
                yield lambda: (self.p_ready.over(t) and (not more or full(self.q_full, t + 1))
                               and (n > 0 or i == 0 or self.acc_free.over(i - 1)))
                product(lambda t=t, n=n: self.s == ("P", t) and self.loaded["do", t % len(self.do_full)] == t
                        and (self.acc is None if n == 0 else self.acc == t - 1), s=("used",))
                self.commit(self.do_empty[t % len(self.do_empty)])
                if more:
                    scores(i, t + 1)
                yield lambda: self.ds_ready.over(t) and (not more or full(self.do_full, t + 1))
                product(lambda t=t: self.dp == ("P", t) and self.loaded["q", t % len(self.q_full)] == t, dp=("used",), acc=t)
                self.commit(self.q_empty[t % len(self.q_empty)])
                if more:
                    dp(i, t + 1)
                    if n + 2 == steps:
                        self.commit(self.kv_empty)
                else:
                    self.commit(self.done)
                t += 1

    def write(self, name, t):
        """A warp's probabilities over its scores."""
        self.wrote[name, t] = self.wrote.get((name, t), 0) + 1
        if self.wrote[name, t] == self.warps:
            setattr(self, name, ("P", t))

    def math(self):
        t = 0
        for i, steps in enumerate(self.items):
            for _ in range(steps):
                slot, turn = t % len(self.do_full), t // len(self.do_full)
                yield lambda: self.do_full[slot].over(turn) and self.s_full.over(t)
                if t % 3 == 0:
                    yield lambda: self.dp_full.over(t)
                    assert self.loaded["do", slot] == t and self.loaded["q", t % len(self.q_full)] == t
                assert self.s == ("S", t)
                yield lambda: True
                self.write("s", t)
                self.p_ready.arrive()
                yield lambda: self.dp_full.over(t)
                assert self.dp == ("S", t) and self.loaded["do", slot] == t  # lse and delta are in the slot
                yield lambda: True
                self.write("dp", t)
                self.ds_ready.arrive()
                self.do_empty[slot].arrive()
                t += 1
            yield lambda: self.done.over(i)
            assert self.acc == t - 1
            yield lambda: True
            self.out += 1
            if self.out == self.warps * (i + 1):
                self.acc = None
            self.acc_free.arrive()


class Queries(Backward):
    """dq. items: key tiles of each. ahead: scores are read a tile ahead (heads of 128)."""

    def __init__(self, items, ahead, warps=3):
        super().__init__(items, warps)
        self.ahead = ahead
        slots = (3, 2) if ahead else (5, 4)
        self.k_full, self.k_empty = ([Barrier(1) for _ in range(slots[0])] for _ in range(2))
        self.v_full, self.v_empty = ([Barrier(1) for _ in range(slots[1])] for _ in range(2))
        self.q_full, self.q_empty, self.s_read = Barrier(2), Barrier(1), Barrier(warps)
        self.dp_full, self.ds_ready = [Barrier(1) for _ in range(2)], [Barrier(warps) for _ in range(2)]
        self.s, self.dp = None, [None, None]
        self.seen, self.wrote = {}, {}

    def roles(self):
        yield "load q", self.load(self.k_full, self.k_empty, "k", True)
        yield "load v", self.load(self.v_full, self.v_empty, "v", False)
        yield "issue", self.issue()
        for w in range(self.warps):
            yield f"math {w}", self.math()

    def load(self, full, empty, name, first):
        t = 0
        for i, tiles in enumerate(self.items):
            if first:
                if i > 0:
                    yield lambda: self.q_empty.over(i - 1)
                self.copy("q", i, self.q_full)
                self.copy("do", i, self.q_full)
            for _ in range(tiles):
                slot, turn = t % len(full), t // len(full)
                if turn > 0:
                    yield lambda: empty[slot].over(turn - 1)
                self.copy((name, slot), t, full[slot])
                t += 1

    def issue(self):
        def full(bars, t):
            return bars[t % len(bars)].over(t // len(bars))

        def scores(i, t, last):
            def s():
                assert self.loaded["q"] == i and self.loaded["k", t % len(self.k_full)] == t
                assert self.s is None, "scores over others"
                self.s = t

            def dp():
                assert self.loaded["do"] == i and self.loaded["v", t % len(self.v_full)] == t
                assert self.dp[t & 1] is None
                self.dp[t & 1] = ("S", t)
            self.pipe.append(s)
            self.commit(self.s_full)
            self.pipe.append(dp)
            self.commit(self.dp_full[t & 1])
            self.commit(self.v_empty[t % len(self.v_empty)])
            if last:
                self.commit(self.q_empty)

        def keys(t):
            return full(self.k_full, t) and full(self.v_full, t)

        def dq(t, j):
            def run():
                assert self.dp[t & 1] == ("P", t) and self.loaded["k", t % len(self.k_full)] == t
                assert self.acc is None if j == 0 else self.acc == t - 1
                self.dp[t & 1], self.acc = None, t
            self.pipe.append(run)

        t = 0
        for i, tiles in enumerate(self.items):
            m = tiles - 1
            yield lambda: self.q_full.over(i) and keys(t)
            scores(i, t, m == 0)
            if self.ahead and m > 0:
                yield lambda: self.s_read.over(i) and keys(t + 1)
                scores(i, t + 1, m == 1)
            for j in range(tiles):
                if not self.ahead and j < m:
                    yield lambda: self.s_read.over(t) and keys(t + 1)
                    scores(i, t + 1, j + 1 == m)
                more = self.ahead and j + 2 <= m
                yield lambda: self.ds_ready[t & 1].over(t >> 1) and (not more or keys(t + 2))
                if j == 0 and i > 0:
                    yield lambda: self.acc_free.over(i - 1)
                dq(t, j)
                self.commit(self.k_empty[t % len(self.k_empty)])
                if j == m:
                    self.commit(self.done)
                if more:
                    scores(i, t + 2, j + 2 == m)
                t += 1

    def math(self):
        def read(t):
            assert self.s == t
            self.seen[t] = self.seen.get(t, 0) + 1
            if self.seen[t] == self.warps:
                self.s = None

        t = 0
        for i, tiles in enumerate(self.items):
            m = tiles - 1
            if self.ahead:
                yield lambda: self.s_full.over(t)
                read(t)
                self.s_read.arrive()
            for j in range(tiles):
                if not self.ahead:
                    yield lambda: self.s_full.over(t)
                    read(t)
                    self.s_read.arrive()
                yield lambda: self.dp_full[t & 1].over(t >> 1)
                assert self.dp[t & 1] == ("S", t)
                yield lambda: True
                self.wrote[t] = self.wrote.get(t, 0) + 1
                if self.wrote[t] == self.warps:
                    self.dp[t & 1] = ("P", t)
                if self.ahead and j < m:
                    yield lambda: self.s_full.over(t + 1)
                    read(t + 1)
                self.ds_ready[t & 1].arrive()
                t += 1
            yield lambda: self.done.over(i)
            assert self.acc == t - 1
            yield lambda: True
            self.out += 1
            if self.out == self.warps * (i + 1):
                self.acc = None
            self.acc_free.arrive()


@pytest.mark.parametrize("make", [lambda n: KeysAndValues(n), lambda n: KeysAndValues(n, (5, 4)), lambda n: Queries(n, True),
                                  lambda n: Queries(n, False)], ids=["dk dv 128", "dk dv 64", "dq 128", "dq 64"])
def test_no_order_of_events_stops_the_backward(make):
    for items in itertools.product((1, 2, 3, 4, 7), repeat=3):
        for choose in orders(8):
            make(items).run(choose)
    rng = random.Random(1)
    for seed in range(60):
        make([rng.randrange(1, 9) for _ in range(8)]).run(at_random(seed))


def test_the_model_finds_a_buffer_that_is_written_too_early():
    """Without the wait for the warps that read the last scores."""
    class Early(Queries):
        def issue(self):
            self.s_read.over = lambda phase: True
            return super().issue()
    with pytest.raises((AssertionError, Stopped)):
        Early((3, 3), False).run(last("math 0"))
