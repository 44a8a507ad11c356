"""The barriers of the kernel for prompts with one gate per head, walked on the CPU.

A wait names a phase by its parity alone: a warp that first looks when two phases are done takes
them for none and waits for ever.  So no phase may follow the one that a warp waits for before
that warp has seen it, however late it looks.  Here each role is a sequence of waits and
arrivals, as in csrc/gla_headgate.cu, and runs under schedules that hold one role back for as long
as any other can go on, and under random ones.  How many barriers take turns, and on which of them
the loads wait, is read from the source.
"""

from __future__ import annotations

import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "chunkwise_linear_rnn_gb300", "csrc",
                      "gla_headgate.cu")
VALUES, SCORES = 2, 2       # warps of these roles; more of them are alike


def read_source():
    """Barriers in turn by name, and whether the loads of the sums alone wait for kDone."""
    with open(SOURCE) as f:
        text = f.read()
    turns = {}
    for name, mark in re.findall(r"constexpr int (k\w+) = \d+;(?: +// (\[\w+\]))?", text):
        turns[name] = mark.strip("[]") or "1"
    loads = text[text.index("load_k(u + 2)"):text.index("load_v(u + 3)")]
    return turns, "!STATE && !wait2(kDone" not in loads


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1


class Kernel:
    """One block's walk over n chunks; `state`: the launch that wants the sums alone; `cut`: the
    last chunk is not full; `deep`: whose rows fall below the floor, by chunk."""

    def __init__(self, n, state, cut, deep, turns, state_loads_wait_done):
        self.n, self.state, self.cut, self.deep = n, state, cut, deep
        self.wait_done = state_loads_wait_done or not state
        slots, sums = (4, 2) if state else (2, 1)
        number = {"slots": slots, "sums": sums, "1": 1, "2": 2, "3": 3}
        self.turns = {k: number[v] for k, v in turns.items()}
        self.slots, self.sums = slots, sums
        count = {"kGFree": VALUES + (0 if state else SCORES), "kPart": VALUES, "kSumFree": VALUES,
                 "kCopy": VALUES, "kP": SCORES, "kOFree": SCORES}
        self.bars = {k: [Barrier(count.get(k, 1)) for _ in range(m)] for k, m in self.turns.items()}
        self.roles = [self.loads(), self.gates(), self.products()]
        self.roles += [self.values() for _ in range(VALUES)]
        if not state:
            self.roles += [self.scores() for _ in range(SCORES)]
        self.waiting = [None for _ in self.roles]      # None: at its beginning

    def wait(self, name, u):
        m = self.turns[name]
        return self.bars[name][u % m], u // m

    def arrive(self, name, u):
        self.bars[name][u % self.turns[name]].arrive()

    # ------------------------------------------------------------ the roles

    def loads(self):
        n, state = self.n, self.state

        def load(name, u):
            if not (state and name == "kFullQ"):
                self.arrive(name, u)
        for u in range(min(n, 3)):
            if u < 2:
                load("kFull", u)
            if u == 0:
                load("kFullQ", 0)
            load("kFullV", u)
        for u in range(n - 1):
            if not state:
                yield self.wait("kQS", u)
            load("kFullQ", u + 1)
            if u + 2 < n:
                yield self.wait("kSum", u)
                load("kFull", u + 2)
            if u + 3 < n:
                if self.wait_done:
                    yield self.wait("kDone", u)
                load("kFullV", u + 3)
        for u in range(max(0, n - 2), n):
            yield self.wait("kFull", u)
        for u in range(max(0, n - 3), n):
            yield self.wait("kFullV", u)
        if not state and n:
            yield self.wait("kFullQ", n - 1)

    def gates(self):
        for u in range(self.n):
            if u >= 2:
                yield self.wait("kGFree", u - 2)
            self.arrive("kGFull", u)

    def part_free(self, j):
        if j >= self.slots:
            yield self.wait("kPartFree", j - self.slots)

    def first_part(self, u):
        yield self.wait("kFullV", u)
        if self.cut and u == self.n - 1:
            yield self.wait("kFull", u)
        yield self.wait("kGFull", u)
        yield from self.part_free(3 * u)
        self.arrive("kGFree", u)
        self.arrive("kPart", 3 * u)

    def values(self):
        n, state = self.n, self.state
        if n and not state:
            self.arrive("kCopy", 0)
        if n:
            yield from self.first_part(0)
        for u in range(n):
            for j in (3 * u + 1, 3 * u + 2):
                yield from self.part_free(j)
                self.arrive("kPart", j)
            if u + 1 < n:
                yield from self.first_part(u + 1)
            yield self.wait("kSum", u)
            self.arrive("kSumFree", u)
            if not state and u + 1 < n:
                yield self.wait("kQS", u)
                self.arrive("kCopy", u + 1)

    def scores(self):
        for u in range(self.n):
            yield self.wait("kGFull", u)
            yield self.wait("kScore", u)
            if self.deep(u):
                yield self.wait("kQS", u)
            self.arrive("kP", u)
            self.arrive("kGFree", u)
            yield self.wait("kDone", u)
            self.arrive("kOFree", u)

    def products(self):
        state, sums = self.state, self.sums
        for u in range(self.n):
            yield self.wait("kFull", u)
            if u >= sums:
                yield self.wait("kSumFree", u - sums)
            for part in range(3):
                yield self.wait("kPart", 3 * u + part)
                self.arrive("kPartFree", 3 * u + part)
                if part or state:
                    continue
                yield self.wait("kFullQ", u)
                if u:
                    yield self.wait("kDone", u - 1)
                self.arrive("kScore", u)
                yield self.wait("kCopy", u)
                if u:
                    yield self.wait("kOFree", u - 1)
                self.arrive("kQS", u)
            self.arrive("kSum", u)
            if state:
                if self.wait_done:
                    self.arrive("kDone", u)
                continue
            yield self.wait("kP", u)
            self.arrive("kDone", u)
        self.arrive("kDrain", 0)
        yield self.wait("kDrain", 0)

    # ------------------------------------------------------------ schedules

    def ready(self, i):
        w = self.waiting[i]
        if w is None:
            return True
        bar, phase = w
        seen = bar.phase % 2 != phase % 2      # what the parity says
        if seen:
            assert bar.phase > phase, "a wait took an earlier phase for its own"
        return seen

    def run(self, order):
        """Lets the first role of `order(n)` that can go on take a step; False when none can."""
        live = set(range(len(self.roles)))
        while live:
            for i in order(len(self.roles)):
                if i in live and self.ready(i):
                    try:
                        self.waiting[i] = next(self.roles[i])
                    except StopIteration:
                        live.remove(i)
                    break
            else:
                return False
        return True


def schedules(roles):
    for late in range(roles):                  # one role only when nothing else can go on
        first = [i for i in range(roles) if i != late]
        yield lambda n, order=[*first, late]: order
        yield lambda n, order=[*first[::-1], late]: order
    for seed in range(20):
        rng = random.Random(seed)
        yield lambda n, rng=rng: rng.sample(range(n), n)


def ends(n, state, cut, turns, wait_done, deep=lambda u: False):
    roles = 3 + VALUES + (0 if state else SCORES)
    return all(Kernel(n, state, cut, deep, turns, wait_done).run(order)
               for order in schedules(roles))


@pytest.mark.parametrize("state", [False, True], ids=["outputs", "sums"])
@pytest.mark.parametrize("cut", [False, True], ids=["full", "cut"])
def test_no_schedule_stops_the_kernel(state, cut):
    turns, wait_done = read_source()
    assert {"kFull", "kSum", "kSumFree", "kDone", "kDrain"} <= set(turns)
    for n in range(14):
        for deep in (lambda u: False, lambda u: True, lambda u: u in (3, 6, 7)):
            assert ends(n, state, cut, turns, wait_done, deep), f"{n} chunks"
            if state:
                break


def test_the_model_sees_a_wait_that_can_be_missed():
    """One barrier for every chunk's sum, and loads of the sums alone that wait for a chunk's end:
    the next phases of both need nothing that the loads have not queued by then."""
    turns, wait_done = read_source()
    assert not ends(9, False, False, {**turns, "kSum": "sums"}, wait_done)
    assert not ends(9, True, False, turns, True)
