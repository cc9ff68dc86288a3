"""What is left when a bounded wait of an attention kernel gives up, simulated
under random schedules: a copy lands later than anybody waits for it. Whoever
gives up sets a flag, waits that find it set give up too, and the block ends;
before it does, somebody has to record the flag, and every copy that was begun
has to have landed, or it lands in the shared memory of another block.

Two orders of the end. "apart": the copying warp leaves by itself and the warps
of arithmetic do (mma.sync kernel over a quantised cache), so both look at the flag after their last
wait. "together": all roles meet, then one looks (tcgen05 kernels). Controls in
which the copying warp alone looks, when its own last copy is begun, must be
seen to fail.
"""

import random

import pytest

from test_attention_protocol_cpu import Barrier, Fault

STAGES = 3


class Sim:
    """A block of n tiles, of which tile `late` lands only when nobody can go on."""

    def __init__(self, n, late, seed, end, looks):
        self.rng = random.Random(seed)
        self.n, self.late, self.end, self.looks = n, late, end, looks
        self.full, self.empty = [Barrier(1) for _ in range(STAGES)], [Barrier(2) for _ in range(STAGES)]
        self.flying, self.gave_up, self.recorded, self.left = [], False, False, 0
        self.waited_out = False

    def wait(self, barrier, parity):
        """Passes, or gives up after the time limit, or soon after somebody did."""
        ok = yield ("wait", barrier, parity)
        if not ok:
            self.gave_up = True
        return ok

    def look(self):
        """At the flag: recorded, and the copies in flight waited for."""
        if self.gave_up:
            self.recorded = True
            yield ("landed",)

    def copies(self):
        for i in range(self.n):
            if i >= STAGES and not (yield from self.wait(self.empty[i % STAGES], (i // STAGES - 1) & 1)):
                break
            self.flying.append(i)
            yield None
        if self.end == "apart" or self.looks == "copies":
            yield from self.look()
        yield from self.leave(self.end == "together")

    def arithmetic(self, w):
        for i in range(self.n):
            yield from self.wait(self.full[i % STAGES], i // STAGES & 1)
            yield None
            if i + STAGES < self.n:
                self.empty[i % STAGES].arrive()
        if self.end == "apart":
            yield ("meet",)
            if w == 0 and self.looks == "all":
                yield from self.look()
        yield from self.leave(False)

    def leave(self, last):
        if self.end == "together":
            yield ("end",)
            if last and self.looks == "all":
                yield from self.look()

    def run(self):
        roles = [self.copies(), self.arithmetic(0), self.arithmetic(1)]
        state, live = [None] * 3, {0, 1, 2}

        def step(w, value=None):
            try:
                state[w] = roles[w].send(value)
            except StopIteration:
                live.discard(w)

        for w in list(live):
            step(w)
        while live:
            choices = []
            for w in live:
                x = state[w]
                if x is None:
                    choices.append((step, w, None))
                elif x[0] == "wait":
                    if x[1].passes(x[2]):
                        choices.append((step, w, True))
                    elif self.gave_up:
                        choices.append((step, w, False))
                elif x[0] == "landed" and not self.flying:
                    choices.append((step, w, None))
            if all(state[w] == ("meet",) for w in (1, 2)) and {1, 2} <= live:
                choices.append((lambda *_: [step(w) for w in (1, 2)], 0, None))
            if all(state[w] == ("end",) for w in live) and len(live) == 3:
                choices.append((lambda *_: [step(w) for w in (1, 2, 0)], 0, None))
            landing = [i for i in self.flying if i != self.late]
            if landing:
                choices.append((self.land, self.rng.choice(landing), None))
            if not choices:
                if self.waited_out:      # in the time of the drain's own limit
                    self.land(self.late)
                    continue
                self.waited_out = True   # the limit has passed: somebody gives up
                w = self.rng.choice([w for w in live if state[w][0] == "wait"])
                step(w, False)
                continue
            f, x, y = self.rng.choice(choices)
            f(x, y)
        if not self.gave_up:
            raise Fault("nobody gave up")
        if not self.recorded:
            raise Fault("given up, and nobody says so")
        if self.flying:
            raise Fault("copies %s land after the block's end" % self.flying)

    def land(self, i, _=None):
        self.flying.remove(i)
        if self.full[i % STAGES].phase == i // STAGES:
            self.full[i % STAGES].arrive()


CASES = [(n, late) for n in (1, 2, 3, 5, 8) for late in range(n)]


@pytest.mark.parametrize("n,late", CASES)
@pytest.mark.parametrize("end", ["apart", "together"])
def test_a_wait_that_gives_up_is_recorded_and_no_copy_outlives_the_block(n, late, end):
    for seed in range(200):
        Sim(n, late, seed, end, "all").run()


@pytest.mark.parametrize("end", ["apart", "together"])
def test_a_look_by_the_copying_warp_alone_fails(end):
    faults = 0
    for n, late in CASES:
        for seed in range(20):
            try:
                Sim(n, late, seed, end, "copies").run()
            except Fault:
                faults += 1
    assert faults > 0
