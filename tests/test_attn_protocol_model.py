"""A CPU model of the bf16 attention kernel's protocol (csrc/gdn_attn_tc.cu): the loader, the
product warp and the two softmax groups as processes over the same ring of tiles, barriers and
in-order tensor pipe.  Random sequences of units must run to their end, every product must read
the tile that it is meant to read, and no stage may be handed back twice."""
from __future__ import annotations

import random

import pytest


class Model:
    """Units are (wide, tiles).  ``keys_first``: a unit's last tiles in the order of the keys.
    ``late``: stages are handed back by the product warp on the softmax's answer, not by the
    softmax when it sees the scores."""

    def __init__(self, units, stages, keys_first=True, late=False, delay=0):
        self.units, self.stages, self.keys_first, self.late, self.delay = units, stages, keys_first, late, delay
        self.full = {}        # load number -> tile
        self.free = {}        # load number -> handed back
        self.loads = 0        # load numbers issued
        self.q_free = [True] + [False] * len(units)
        self.q_full = [False] * len(units)
        self.scores = ([], [])   # per X: (unit, tile, stages freed) whose scores are done
        self.ready = [0, 0]      # weights ready, counted
        self.outs = ([], [])     # per X: (unit, last) outputs done

    def last_order(self, left):
        order = [0, 1]
        if self.keys_first and left[1] is not None and (left[0] is None or left[1] < left[0]):
            order = [1, 0]
        return [x for x in order if left[x] is not None]

    # -- the loader
    def load(self, tile):
        n = self.loads
        while n >= self.stages and not self.free.get(n - self.stages):
            yield
        self.full[n] = tile
        self.loads += 1

    def loader(self):
        left, shared, old = [None, None], False, None
        for i, (wide, n) in enumerate(self.units + [(None, 0)]):
            def values(x):
                if not (shared and x == 1):
                    yield from self.load((old, "v", left[x]))
                left[x] = None
            order = self.last_order(left)
            if order and order[0] == 1:
                yield from values(1)
            if left[0] is not None:
                yield from values(0)
            if wide is None:
                if left[1] is not None:
                    yield from values(1)
                return
            while not self.q_free[i]:
                yield
            self.q_full[i] = True
            yield from self.load((i, "k", 0))
            if left[1] is not None:
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

    # -- the products
    def next_tile(self, want):
        n = self.used
        while n not in self.full:
            yield
        assert self.full[n] == want, (n, self.full[n], want)
        self.used += 1
        return n

    def products(self):
        self.used = 0
        left, shared, old, shared_v = [None, None], False, None, None
        held, answers = ([], []), [0, 0]

        def scores(x, unit, tile, freed):
            self.scores[x].append((unit, tile, freed))
            held[x].extend(freed)

        def weights(x):
            answers[x] += 1
            while self.ready[x] < answers[x]:
                yield
            if self.late:
                for n in held[x]:
                    self.free[n] = True
                held[x].clear()

        def last_output(x):
            nonlocal shared_v
            if not (shared and x == 1):
                shared_v = yield from self.next_tile((old, "v", left[x]))
            yield from weights(x)
            self.outs[x].append((old, True))
            if not shared or x == 1:
                self.free[shared_v] = True
            left[x] = None

        for i, (wide, n) in enumerate(self.units + [(None, 0)]):
            order = self.last_order(left)
            if order and order[0] == 1:
                yield from last_output(1)
            if left[0] is not None:
                yield from last_output(0)
            if wide is None:
                if left[1] is not None:
                    yield from last_output(1)
                return
            while not self.q_full[i]:
                yield
            k = yield from self.next_tile((i, "k", 0))
            scores(0, i, 0, [] if wide else [k])
            if left[1] is not None:
                yield from last_output(1)
            if wide:
                scores(1, i, 0, [k])
                for t in range(n - 1):
                    v = yield from self.next_tile((i, "v", t))
                    yield from weights(0)
                    k_next = yield from self.next_tile((i, "k", t + 1))
                    scores(0, i, t + 1, [])
                    yield from weights(1)
                    scores(1, i, t + 1, [k_next, v])
                left = [n - 1, n - 1]
            else:
                if n > 1:
                    k = yield from self.next_tile((i, "k", 1))
                    scores(1, i, 1, [k])
                for t in range(2, n):
                    x = t & 1
                    v = yield from self.next_tile((i, "v", t - 2))
                    yield from weights(x)
                    k = yield from self.next_tile((i, "k", t))
                    scores(x, i, t, [k, v])
                odd = (n - 1) & 1
                left = [n - 1 - odd, n - 2 + odd if n > 1 else None]
            self.q_free[i + 1] = True
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
                if not self.late:
                    for n_load in self.scores[x][seen][2]:
                        assert not self.free.get(n_load)
                        self.free[n_load] = True
                for _ in range(random.randint(0, self.delay)):
                    yield
                seen += 1
                self.ready[x] += 1
            both = not wide and n > 1
            for y in ((0, 1) if both else (x,)):
                while tiles and (i, True) not in self.outs[y]:
                    yield

    def run(self):
        procs = [self.loader(), self.products(), self.softmax(0), self.softmax(1)]
        idle = 0
        while procs:
            before = (self.loads, getattr(self, "used", 0), len(self.scores[0]), len(self.scores[1]),
                      tuple(self.ready), len(self.outs[0]), len(self.outs[1]), len(self.free), len(procs))
            for p in list(procs):
                try:
                    next(p)
                except StopIteration:
                    procs.remove(p)
            after = (self.loads, getattr(self, "used", 0), len(self.scores[0]), len(self.scores[1]),
                     tuple(self.ready), len(self.outs[0]), len(self.outs[1]), len(self.free), len(procs))
            idle = idle + 1 if before == after else 0
            if idle > 10 + 4 * self.delay:
                return False
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
    """Handing stages back on the softmax's answer, with a unit's last tiles in the order of the
    X, an odd number of tiles leaves the ring waiting for a stage that is handed back only after
    the tile that waits for it."""
    units = [(False, 3), (False, 3)]
    assert not Model(units, 5, keys_first=False, late=True).run()
    assert Model(units, 5, keys_first=True, late=True).run()
    assert Model(units, 5).run()
