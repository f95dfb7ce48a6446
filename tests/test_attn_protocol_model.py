"""A CPU model of the bf16 attention kernel's protocol (csrc/gdn_attn_tc.cu): the loader, the two
product warps and the two softmax groups as processes over the same ring of tiles.  Its barriers
know a phase's parity only, as the hardware's do, and loads arrive late and out of order.  Random
sequences of units must run to their end, every product must read the tile that it is meant to
read, and a stage must have been handed back twice (once by each X, or twice by the one X that
reads it) before it is filled again."""
from __future__ import annotations

import random

import pytest


class Wrong(Exception):
    """A product read another tile than it should, or a stage was handed back too often."""


class Model:
    """Units are (wide, tiles).  ``arrivals``: how often a stage is handed back before the loader
    fills it again (2 in the kernel).  ``skip``: a product warp does not wait for the other X's
    tiles."""

    def __init__(self, units, stages, delay=0, late=0, arrivals=2, skip=False):
        self.units, self.stages, self.delay, self.late = units, stages, delay, late
        self.arrivals, self.skip = arrivals, skip
        self.filled = [0] * stages      # fillings of a stage that have arrived
        self.content = [None] * stages  # what is in it; None while a filling is under way
        self.freed = [0] * stages       # how often it was handed back
        self.flying = []                # [steps left, stage, tile]
        self.loads = 0
        self.q_free = [2] + [0] * len(units)
        self.q_full = [False] * len(units)
        self.scores = ([], [])          # per X: (unit, tile, stages freed, wide) whose scores are done
        self.ready = [0, 0]             # weights ready, counted
        self.outs = (set(), set())      # per X: units whose last output is done
        self.met = [0, 0]
        self.steps = 0

    def hand_back(self, stage, times):
        self.freed[stage] += times
        if self.freed[stage] > 2 * self.filled[stage]:
            raise Wrong("handed back too often")
        self.steps += 1

    # -- the loader
    def load(self, tile):
        stage, turn = self.loads % self.stages, self.loads // self.stages
        # waits for the phase before `turn` of "empty", by parity
        while (self.freed[stage] // self.arrivals) & 1 == (turn & 1) ^ 1:
            yield
        if self.freed[stage] < 2 * turn:
            raise Wrong("filled while it is read")
        self.content[stage] = None
        self.flying.append([random.randint(0, self.late), stage, tile])
        self.loads += 1

    def arrive(self):
        for f in list(self.flying):
            f[0] -= 1
            if f[0] < 0:
                self.flying.remove(f)
                self.content[f[1]] = f[2]
                self.filled[f[1]] += 1
                self.steps += 1

    def loader(self):
        left, shared, old = [None, None], False, None
        for i, (wide, n) in enumerate(self.units + [(None, 0)]):
            def values(x):
                if left[x] is not None and not (shared and x == 1):
                    yield from self.load((old, "v", left[x]))
                left[x] = None
            if left[1] is not None and left[1] < left[0]:
                yield from values(1)
            yield from values(0)
            if wide is None:
                yield from values(1)
                return
            while self.q_free[i] < 2:
                yield
            self.q_full[i] = True
            yield from self.load((i, "k", 0))
            yield from values(1)
            if wide:
                for t in range(n - 1):
                    yield from self.load((i, "v", t))
                    yield from self.load((i, "k", t + 1))
                left = [n - 1, n - 1]
            else:
                if n > 1:
                    yield from self.load((i, "k", 1))
                for t in range(2, n):
                    yield from self.load((i, "v", t - 2))
                    yield from self.load((i, "k", t))
                odd = (n - 1) & 1
                left = [n - 1 - odd, n - 2 + odd if n > 1 else None]
            shared, old = wide, i

    # -- the products of one X
    def products(self, x):
        ring = 0
        left, shared, old = [None, None], False, None
        answers = 0

        def tile(want, mine):
            """The next tile of the ring; ``mine``: this X reads it."""
            nonlocal ring
            stage, turn = ring % self.stages, ring // self.stages
            ring += 1
            if mine or not self.skip:
                while self.filled[stage] & 1 == turn & 1:
                    yield
            if mine and self.content[stage] != want:
                raise Wrong((self.content[stage], want))
            return stage

        def check(stage, want):
            if self.content[stage] != want:
                raise Wrong((self.content[stage], want))

        def output():
            nonlocal answers
            answers += 1
            while self.ready[x] < answers:
                yield

        def last_output(stage, t):
            yield from output()
            check(stage, (old, "v", t))
            self.hand_back(stage, 1 if shared else 2)
            self.outs[x].add(old)

        for i, (wide, n) in enumerate(self.units + [(None, 0)]):
            if left[1] is not None and not shared and left[1] < left[0]:
                v = yield from tile((old, "v", left[1]), x == 1)
                if x == 1:
                    yield from last_output(v, left[1])
                left[1] = None
            if left[0] is not None:
                mine = x == 0 or shared
                v = yield from tile((old, "v", left[0]), mine)
                if mine:
                    yield from last_output(v, left[0])
                if shared:
                    left[1] = None
                left[0] = None
            if wide is not None:
                k = yield from tile((i, "k", 0), wide or x == 0)
                while not self.q_full[i]:
                    yield
                if x == 0:
                    self.scores[0].append((i, 0, [k], wide))
            if left[1] is not None:
                v = yield from tile((old, "v", left[1]), x == 1)
                if x == 1:
                    yield from last_output(v, left[1])
                left[1] = None
            if wide is None:
                return
            if wide:
                if x == 1:
                    check(k, (i, "k", 0))
                    self.scores[1].append((i, 0, [k], wide))
                for t in range(n - 1):
                    v = yield from tile((i, "v", t), True)
                    k = yield from tile((i, "k", t + 1), True)
                    yield from output()
                    check(v, (i, "v", t))
                    check(k, (i, "k", t + 1))
                    self.scores[x].append((i, t + 1, [k, v], wide))
                left = [n - 1, n - 1]
            else:
                if n > 1:
                    k = yield from tile((i, "k", 1), x == 1)
                    if x == 1:
                        self.scores[1].append((i, 1, [k], wide))
                for t in range(2, n):
                    mine = t & 1 == x
                    v = yield from tile((i, "v", t - 2), mine)
                    k = yield from tile((i, "k", t), mine)
                    if not mine:
                        continue
                    yield from output()
                    check(v, (i, "v", t - 2))
                    check(k, (i, "k", t))
                    self.scores[x].append((i, t, [k, v], wide))
                odd = (n - 1) & 1
                left = [n - 1 - odd, n - 2 + odd if n > 1 else None]
            self.q_free[i + 1] += 1
            shared, old = wide, i

    # -- the softmax of one X
    def softmax(self, x):
        seen = 0
        for i, (wide, n) in enumerate(self.units):
            tiles = range(n) if wide else range(x, n, 2)
            for t in tiles:
                while len(self.scores[x]) <= seen:
                    yield
                assert self.scores[x][seen][:2] == (i, t)
                for stage in self.scores[x][seen][2]:
                    self.hand_back(stage, 1 if wide else 2)
                for _ in range(random.randint(0, self.delay)):
                    yield
                seen += 1
                self.ready[x] += 1
            while tiles and i not in self.outs[x]:
                yield
            if not wide and n > 1:  # both X meet to join their outputs
                self.met[x] += 1
                while self.met[x ^ 1] < self.met[x]:
                    yield

    def run(self):
        procs = [self.loader(), self.products(0), self.products(1), self.softmax(0), self.softmax(1)]
        idle, before = 0, None
        while procs:
            self.arrive()
            random.shuffle(procs)
            for p in list(procs):
                try:
                    next(p)
                except StopIteration:
                    procs.remove(p)
            after = (self.loads, len(self.scores[0]), len(self.scores[1]), tuple(self.ready),
                     len(self.outs[0]), len(self.outs[1]), self.steps, tuple(self.met), len(procs))
            idle = idle + 1 if before == after and not self.flying else 0
            before = after
            if idle > 10 + 4 * self.delay:
                return False
        return True


def random_units(rng):
    return [(rng.random() < 0.4, rng.choice((1, 1, 2, 3, 4, 5, 6, 7, 11))) for _ in range(rng.randint(1, 9))]


@pytest.mark.parametrize("stages", [5, 10])
def test_every_sequence_of_units_ends(stages):
    rng = random.Random(stages)
    random.seed(stages)
    for trial in range(2000):
        units = random_units(rng)
        assert Model(units, stages, delay=trial % 5, late=(0, 3, 30)[trial % 3]).run(), units


def test_model_finds_a_deadlock():
    """Too few stages for what the two X hold at once; a stage that waits for an arrival that
    nobody makes."""
    units = [(False, 3), (False, 3)]
    random.seed(1)
    assert not Model(units, 1).run()
    assert not Model(units, 5, arrivals=3).run()
    assert Model(units, 5).run()


def test_model_finds_a_wait_for_the_wrong_filling():
    """A product warp that passes over the other X's tiles without waiting for them takes a
    stage's filling before last for its own when loads arrive out of order."""
    random.seed(2)
    wrong = 0
    for _ in range(300):
        try:
            if not Model([(False, 11)] * 4, 5, delay=2, late=30, skip=True).run():
                wrong += 1
        except Wrong:
            wrong += 1
    assert wrong > 0
