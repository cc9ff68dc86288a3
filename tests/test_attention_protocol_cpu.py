"""The hand-over of tiles between the warps of the tcgen05 attention kernel,
simulated under random schedules: copies of keys, values and q that land in
any order and late, two streams of products whose ends come late, and two
groups of weights. Barriers have the hardware's rule: a wait for a parity
passes when the barrier's current phase has the other one, so a waiter that
passes over a phase can be let through too early or held for ever.

The kernel numbers the barriers of a tile j by j % 6 (its stage j % 3 and its
stream j % 2). The control numbers them by the stage alone, and must be seen
to fail.
"""

import random

import pytest

STAGES, SLOTS = 3, 6


class Fault(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending < 0:
            raise Fault("one arrival too many")
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passes(self, parity):
        return (self.phase & 1) != parity


class Sim:
    """items: tiles of each item of a block's run. number(j): a tile's barrier."""

    def __init__(self, items, seed, number, slots):
        self.rng = random.Random(seed)
        self.number, self.slots = number, slots
        self.tiles = [(i, t) for i, n in enumerate(items) for t in range(n)]
        self.last = {}
        for j, (i, _) in enumerate(self.tiles):
            self.last[i] = j
        n = slots
        self.k_full, self.k_empty = [Barrier(1) for _ in range(n)], [Barrier(1) for _ in range(n)]
        self.v_full, self.v_empty = [Barrier(1) for _ in range(n)], [Barrier(1) for _ in range(n)]
        self.q_full, self.q_empty = Barrier(1), Barrier(2)
        self.s_full, self.p_half, self.p_three, self.p_full, self.pv_done = (
            [Barrier(1), Barrier(1)] for _ in range(5))
        self.k, self.v = [None] * STAGES, [None] * STAGES   # tile whose data a stage holds
        self.q, self.k_issued = None, 0
        self.scores = [None, None]
        self.summed = []
        self.events = []          # things that happen later, in any order (or in order, per queue)
        self.queues = {0: [], 1: []}

    def phase(self, j):
        return (j // self.slots) & 1

    # --- the warps, as generators: `yield (barrier, parity)` waits
    def copies(self, data, empty, what):
        """Keys, and values: one warp, but each side goes on whenever it can."""
        for j in range(len(self.tiles)):
            b = j - STAGES
            if b >= 0:
                yield empty[self.number(b)], self.phase(b)
            if what == "v" and self.k_issued <= j:
                yield lambda j=j: self.k_issued > j
            if what == "k":
                self.k_issued = j + 1
            data[j % STAGES] = None
            self.events.append((what, j))

    def q_copies(self):
        n = 0
        for j, (i, t) in enumerate(self.tiles):
            if t == 0 or j == 0:
                if n:
                    yield self.q_empty, (n - 1) & 1
                self.q = None
                self.events.append(("q", i))
                n += 1

    def products(self, s):
        n = 0
        for item, i in enumerate(sorted(self.last)):
            jb = self.last[i] + 1
            mine = [j for j, (k, _) in enumerate(self.tiles) if k == i and j % 2 == s]
            yield self.q_full, item & 1
            if not mine and jb < len(self.tiles):
                self.q_empty.arrive()
            for j in mine:
                yield self.k_full[self.number(j)], self.phase(j)
                if n:
                    yield self.pv_done[s], (n - 1) & 1
                if self.k[j % STAGES] != j or self.q != i:
                    raise Fault("scores of tile %d from %s, q of %s" % (j, self.k[j % STAGES], self.q))
                todo = [("scores", s, j), ("arrive", self.s_full[s])]
                if j + STAGES < len(self.tiles):
                    todo.append(("arrive", self.k_empty[self.number(j)]))
                if j + 2 >= jb and jb < len(self.tiles):
                    todo.append(("arrive", self.q_empty))
                self.queues[s] += todo
                yield self.v_full[self.number(j)], self.phase(j)
                yield self.p_half[s], n & 1
                yield self.p_three[s], n & 1
                yield self.p_full[s], n & 1
                if self.v[j % STAGES] != j:
                    raise Fault("sums of tile %d from %s" % (j, self.v[j % STAGES]))
                todo = [("sums", s, j), ("arrive", self.pv_done[s])]
                if j + STAGES < len(self.tiles):
                    todo.append(("arrive", self.v_empty[self.number(j)]))
                self.queues[s] += todo
                n += 1

    def weights(self, s):
        n = 0
        for i in sorted(self.last):
            mine = [j for j, (k, _) in enumerate(self.tiles) if k == i and j % 2 == s]
            yield "meet"
            for j in mine:
                yield self.s_full[s], n & 1
                yield self.v_full[self.number(j)], self.phase(j)
                if self.scores[s] != j or self.v[j % STAGES] != j:
                    raise Fault("weights of tile %d from %s, %s" % (j, self.scores[s], self.v[j % STAGES]))
                self.p_half[s].arrive()
                yield None
                self.p_three[s].arrive()
                yield None
                self.p_full[s].arrive()
                n += 1
            if mine:
                yield self.pv_done[s], (n - 1) & 1
            yield "meet"
            yield "meet"

    def happen(self):
        """One of the pending copies or products ends."""
        choices = [("event", k) for k in range(len(self.events))] + [("queue", s) for s in (0, 1) if self.queues[s]]
        if not choices:
            return False
        kind, k = self.rng.choice(choices)
        if kind == "event":
            what, x = self.events.pop(k)
            if what == "q":
                self.q = x
                self.q_full.arrive()
            else:
                (self.k if what == "k" else self.v)[x % STAGES] = x
                (self.k_full if what == "k" else self.v_full)[self.number(x)].arrive()
        else:
            todo = self.queues[k].pop(0)
            if todo[0] == "arrive":
                todo[1].arrive()
            elif todo[0] == "scores":
                self.scores[todo[1]] = todo[2]
            else:
                self.summed.append(todo[2])
        return True

    def run(self):
        warps = [self.copies(self.k, self.k_empty, "k"), self.q_copies(), self.products(0), self.products(1),
                 self.weights(0), self.weights(1), self.copies(self.v, self.v_empty, "v")]
        waits = [None] * 7
        live = set(range(7))
        met = set()
        slow = self.rng.choice([None, 0, 1, 2, 3, 4, 5, 6])    # a warp that gets few turns
        while live:
            ready = [w for w in live if waits[w] is None or (callable(waits[w]) and waits[w]()) or
                     (isinstance(waits[w], tuple) and waits[w][0].passes(waits[w][1]))]
            if slow in ready and len(ready) > 1 and self.rng.random() < 0.9:
                ready.remove(slow)
            if (not ready or self.rng.random() < 0.4) and self.happen():
                continue
            if not ready:
                raise Fault("nobody can go on")
            w = self.rng.choice(ready)
            try:
                waits[w] = next(warps[w])
                if waits[w] == "meet":
                    met.add(w)
                    if met == {4, 5}:
                        waits[4] = waits[5] = None
                        met = set()
            except StopIteration:
                live.discard(w)
        while self.happen():
            pass
        if sorted(self.summed) != list(range(len(self.tiles))):
            raise Fault("sums missing")


SHAPES = [[1], [2], [3], [1, 1], [1, 1, 1, 1, 1], [7], [8, 1, 1, 5], [1, 2, 3, 4], [20], [4, 9, 2], [2, 2, 2, 2, 2]]


@pytest.mark.parametrize("items", SHAPES)
def test_every_tile_is_summed_once_from_its_own_data(items):
    for seed in range(300):
        Sim(items, seed, lambda j: j % SLOTS, SLOTS).run()


def test_barriers_numbered_by_the_stage_alone_fail():
    """Control: with a barrier a stage, a stream passes over the phases of the
    other stream's tiles."""
    faults = 0
    for seed in range(400):
        try:
            Sim([20], seed, lambda j: j % STAGES, STAGES).run()
        except Fault:
            faults += 1
    assert faults > 0
