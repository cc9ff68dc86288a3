"""The hand-over of tiles between the warps of the tcgen05 kernel that attends
over 4 bits, simulated under random schedules: copies of codes that land in any
order, a group of warps for each stream that turns codes into keys and values
(and q at an item's begin), two streams of products whose ends come late, and
two groups of weights. Barriers have the hardware's rule: a wait for a parity
passes when the barrier's current phase has the other one.

Three controls must be seen to fail: codes' barriers numbered by the stage
alone, and one barrier for the end of an item's q, waited for by the group that
writes the next one, or by both (one of them can be lapped, and is held for
ever).
"""

import random

import pytest

from test_attention_protocol_cpu import SHAPES, Barrier, Fault

STAGES, SLOTS = 3, 6


class Sim:
    """items: tiles of each item of a block's run. number(j): the barrier of tile j's codes."""

    def __init__(self, items, seed, number=lambda j: j % SLOTS, slots=SLOTS, q_ends="own"):
        self.rng = random.Random(seed)
        self.number, self.slots, self.q_ends = number, slots, q_ends
        self.tiles = [(i, t) for i, n in enumerate(items) for t in range(n)]
        self.last = {i: j for j, (i, _) in enumerate(self.tiles)}
        two = lambda: [Barrier(1), Barrier(1)]  # noqa: E731
        self.c_full, self.c_empty = [Barrier(1) for _ in range(slots)], [Barrier(1) for _ in range(slots)]
        self.k_full, self.k_empty, self.v_full, self.v_empty = two(), two(), two(), two()
        self.q_full, self.q_empty = Barrier(1), [Barrier(2), Barrier(2)]
        self.s_full, self.p_half, self.p_three, self.p_full, self.pv_done = two(), two(), two(), two(), two()
        self.words_full = [two(), two()]
        self.codes = [None] * STAGES
        self.k, self.v, self.scores, self.q = [None, None], [None, None], [None, None], None
        self.words = [[None, None], [None, None]]
        self.summed = []
        self.events, self.queues = [], {0: [], 1: []}

    def phase(self, j):
        return (j // self.slots) & 1

    def copies(self):
        for j in range(len(self.tiles)):
            b = j - STAGES
            if b >= 0:
                yield self.c_empty[self.number(b)], self.phase(b)
            self.codes[j % STAGES] = None
            self.events.append(j)

    def unpack(self, s):
        n_items = n_ends = 0
        for j, (i, t) in enumerate(self.tiles):
            own = j % 2 == s
            if t == 0 or j == 0:
                if n_items and self.q_ends == "own":
                    if own:
                        yield self.q_empty[s], n_ends & 1
                        n_ends += 1
                elif n_items and (own or self.q_ends == "both"):
                    yield self.q_empty[0], (n_items - 1) & 1
                n_items += 1
                if own:
                    self.q = None
                    yield None
                    self.q = i
                    self.q_full.arrive()
            if not own:
                continue
            use = j // 2
            yield self.c_full[self.number(j)], self.phase(j)
            if use:
                yield self.k_empty[s], (use - 1) & 1
            self.words[s][use & 1] = j
            self.words_full[s][use & 1].arrive()
            self.k[s] = None
            yield None
            if self.codes[j % STAGES] != j:
                raise Fault("keys of tile %d from %s" % (j, self.codes[j % STAGES]))
            self.k[s] = j
            self.k_full[s].arrive()
            if use:
                yield self.v_empty[s], (use - 1) & 1
            self.v[s] = None
            yield None
            if self.codes[j % STAGES] != j:
                raise Fault("values of tile %d from %s" % (j, self.codes[j % STAGES]))
            self.v[s] = j
            self.v_full[s].arrive()
            if j + STAGES < len(self.tiles):
                self.c_empty[self.number(j)].arrive()

    def products(self, s):
        n = 0
        for item, i in enumerate(sorted(self.last)):
            jb = self.last[i] + 1
            mine = [j for j, (k, _) in enumerate(self.tiles) if k == i and j % 2 == s]
            yield self.q_full, item & 1
            if not mine and jb < len(self.tiles):
                self.q_empty[jb & 1 if self.q_ends == "own" else 0].arrive()
            for j in mine:
                yield self.k_full[s], n & 1
                if n:
                    yield self.pv_done[s], (n - 1) & 1
                todo = [("scores", j, i), ("arrive", self.s_full[s])]
                if j + 2 < len(self.tiles):
                    todo.append(("arrive", self.k_empty[s]))
                if j + 2 >= jb and jb < len(self.tiles):
                    todo.append(("arrive", self.q_empty[jb & 1 if self.q_ends == "own" else 0]))
                self.queues[s] += todo
                yield self.v_full[s], n & 1
                yield self.p_half[s], n & 1
                yield self.p_three[s], n & 1
                yield self.p_full[s], n & 1
                todo = [("sums", j, i), ("arrive", self.pv_done[s])]
                if j + 2 < len(self.tiles):
                    todo.append(("arrive", self.v_empty[s]))
                self.queues[s] += todo
                n += 1

    def weights(self, s):
        n = 0
        for i in sorted(self.last):
            mine = [j for j, (k, _) in enumerate(self.tiles) if k == i and j % 2 == s]
            yield "meet"
            for j in mine:
                yield self.s_full[s], n & 1
                yield self.words_full[s][n & 1], (n >> 1) & 1
                for barrier in (self.p_half[s], self.p_three[s], self.p_full[s]):
                    if self.scores[s] != j or self.words[s][n & 1] != j:
                        raise Fault("weights of tile %d from %s, %s" % (j, self.scores[s], self.words[s]))
                    barrier.arrive()
                    yield None
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
            j = self.events.pop(k)
            self.codes[j % STAGES] = j
            self.c_full[self.number(j)].arrive()
            return True
        todo = self.queues[k].pop(0)
        if todo[0] == "arrive":
            todo[1].arrive()
        elif todo[0] == "scores":       # reads q and the keys until now
            if self.k[k] != todo[1] or self.q != todo[2]:
                raise Fault("scores of tile %d from %s, q of %s" % (todo[1], self.k[k], self.q))
            self.scores[k] = todo[1]
        else:
            if self.v[k] != todo[1]:
                raise Fault("sums of tile %d from %s" % (todo[1], self.v[k]))
            self.summed.append(todo[1])
        return True

    def run(self):
        warps = [self.copies(), self.unpack(0), self.unpack(1), self.products(0), self.products(1), self.weights(0),
                 self.weights(1)]
        waits = [None] * len(warps)
        live, met = set(range(len(warps))), set()
        slow = self.rng.choice([None] + list(live))    # warps that get few turns
        while live:
            ready = [w for w in live if waits[w] is None or
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
                    if met == {5, 6}:
                        waits[5] = waits[6] = None
                        met = set()
            except StopIteration:
                live.discard(w)
        while self.happen():
            pass
        if sorted(self.summed) != list(range(len(self.tiles))):
            raise Fault("sums missing")


MORE = SHAPES + [[1] * 12, [1, 2] * 5, [3, 1, 1, 1, 2, 1, 1]]


@pytest.mark.parametrize("items", MORE)
def test_every_tile_is_summed_once_from_its_own_data(items):
    for seed in range(300):
        Sim(items, seed).run()


def faults(items, **kw):
    n = 0
    for seed in range(600):
        try:
            Sim(items, seed, **kw).run()
        except Fault:
            n += 1
    return n


def test_codes_numbered_by_the_stage_alone_fail():
    assert faults([20], number=lambda j: j % STAGES, slots=STAGES) > 0


@pytest.mark.parametrize("q_ends", ["writer", "both"])
def test_one_barrier_for_the_end_of_q_fails(q_ends):
    assert sum(faults(items, q_ends=q_ends) for items in ([1, 2] * 6, [1] * 12, [3, 1, 1, 1, 2, 1, 1] * 2)) > 0
