"""A CPU model of the bf16 attention kernel's protocol (csrc/gdn_attn_tc.cu): the loader, the two
product warps and the two softmax groups as processes over the same ring of tiles and barriers.
Random sequences of units must run to their end, every product must read the tile that it is
meant to read, and each stage must be handed back twice (once by each X, or twice by the one X
that reads it) before it is filled again."""
from __future__ import annotations

import random

import pytest


class Model:
    """Units are (wide, tiles).  ``arrivals``: how often a stage is handed back before the loader
    fills it again (2 in the kernel)."""

    def __init__(self, units, stages, delay=0, arrivals=2):
        self.units, self.stages, self.delay, self.arrivals = units, stages, delay, arrivals
        self.full = {}           # load number -> tile
        self.free = {}           # load number -> arrivals
        self.loads = 0           # load numbers issued
        self.q_free = [2] + [0] * len(units)
        self.q_full = [False] * len(units)
        self.scores = ([], [])   # per X: (unit, tile, loads freed) whose scores are done
        self.ready = [0, 0]      # weights ready, counted
        self.outs = (set(), set())  # per X: units whose last output is done
        self.steps = 0

    def hand_back(self, n, times):
        self.free[n] = self.free.get(n, 0) + times
        assert self.free[n] <= 2, n
        self.steps += 1

    # -- the loader
    def load(self, tile):
        n = self.loads
        while n >= self.stages and self.free.get(n - self.stages, 0) < self.arrivals:
            yield
        self.full[n] = tile
        self.loads += 1

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

        def tile(n, want):
            while n not in self.full:
                yield
            assert self.full[n] == want, (n, self.full[n], want)

        def output():
            nonlocal answers
            answers += 1
            while self.ready[x] < answers:
                yield

        def last_output(n, t):
            yield from tile(n, (old, "v", t))
            yield from output()
            self.hand_back(n, 1 if shared else 2)
            self.outs[x].add(old)

        for i, (wide, n) in enumerate(self.units + [(None, 0)]):
            if left[1] is not None and not shared and left[1] < left[0]:
                ring += 1
                if x == 1:
                    yield from last_output(ring - 1, left[1])
                left[1] = None
            if left[0] is not None:
                ring += 1
                if x == 0 or shared:
                    yield from last_output(ring - 1, left[0])
                if shared:
                    left[1] = None
                left[0] = None
            if wide is not None:
                k, ring = ring, ring + 1
                while not self.q_full[i]:
                    yield
                if x == 0:
                    yield from tile(k, (i, "k", 0))
                    self.scores[0].append((i, 0, [k], wide))
            if left[1] is not None:
                ring += 1
                if x == 1:
                    yield from last_output(ring - 1, left[1])
                left[1] = None
            if wide is None:
                return
            if wide:
                if x == 1:
                    yield from tile(k, (i, "k", 0))
                    self.scores[1].append((i, 0, [k], wide))
                for t in range(n - 1):
                    v, k, ring = ring, ring + 1, ring + 2
                    yield from tile(v, (i, "v", t))
                    yield from output()
                    yield from tile(k, (i, "k", t + 1))
                    self.scores[x].append((i, t + 1, [k, v], wide))
                left = [n - 1, n - 1]
            else:
                if n > 1:
                    k, ring = ring, ring + 1
                    if x == 1:
                        yield from tile(k, (i, "k", 1))
                        self.scores[1].append((i, 1, [k], wide))
                for t in range(2, n):
                    v, k, ring = ring, ring + 1, ring + 2
                    if t & 1 != x:
                        continue
                    yield from tile(v, (i, "v", t - 2))
                    yield from output()
                    yield from tile(k, (i, "k", t))
                    self.scores[x].append((i, t, [k, v], wide))
                odd = (n - 1) & 1
                left = [n - 1 - odd, n - 2 + odd if n > 1 else None]
            self.q_free[i + 1] += 1
            shared, old = wide, i

    # -- the softmax of one X
    def softmax(self, x):
        seen = 0
        met = self.met
        for i, (wide, n) in enumerate(self.units):
            tiles = range(n) if wide else range(x, n, 2)
            for t in tiles:
                while len(self.scores[x]) <= seen:
                    yield
                assert self.scores[x][seen][:2] == (i, t)
                for n_load in self.scores[x][seen][2]:
                    self.hand_back(n_load, 1 if wide else 2)
                for _ in range(random.randint(0, self.delay)):
                    yield
                seen += 1
                self.ready[x] += 1
            while tiles and i not in self.outs[x]:
                yield
            if not wide and n > 1:  # both X meet to join their outputs
                met[x] += 1
                while met[x ^ 1] < met[x]:
                    yield

    def run(self):
        self.met = [0, 0]
        procs = [self.loader(), self.products(0), self.products(1), self.softmax(0), self.softmax(1)]
        idle, before = 0, None
        while procs:
            for p in list(procs):
                try:
                    next(p)
                except StopIteration:
                    procs.remove(p)
            after = (self.loads, len(self.scores[0]), len(self.scores[1]), tuple(self.ready),
                     len(self.outs[0]), len(self.outs[1]), self.steps, tuple(self.met), len(procs))
            idle = idle + 1 if before == after else 0
            before = after
            if idle > 10 + 4 * self.delay:
                return False
        assert all(v == 2 for v in self.free.values())
        return True


def random_units(rng):
    return [(rng.random() < 0.4, rng.choice((1, 1, 2, 3, 4, 5, 6, 7, 11))) for _ in range(rng.randint(1, 9))]


@pytest.mark.parametrize("stages", [5, 10])
def test_every_sequence_of_units_ends(stages):
    rng = random.Random(stages)
    random.seed(stages)
    for trial in range(1500):
        units = random_units(rng)
        assert Model(units, stages, delay=trial % 5).run(), units


def test_model_finds_a_deadlock():
    """Too few stages for what the two X hold at once, and a stage that waits for an arrival that
    nobody makes."""
    units = [(False, 3), (False, 3)]
    assert not Model(units, 1).run()
    assert not Model(units, 5, arrivals=3).run()
    assert Model(units, 5).run()
