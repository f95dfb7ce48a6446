"""A CPU model of the tensor-core kernel's protocol over an 8-bit cache (csrc/gdn_attn_tc.cu): that
over a bf16 cache (tests/test_attn_protocol_model.py) with the four warps that turn loaded tiles, and
a unit's queries, into fp16 between the loads and the products.  Loads, and the scales that come
with key tiles, arrive late and out of order; barriers know a phase's parity only.  Random sequences
of units must end, every product must read its tile turned, and every tile must be turned with its
own scales."""
from __future__ import annotations

import random

import pytest

from tests.test_attn_protocol_model import Model, Wrong, random_units

TURNERS = 4


class Queries:
    """Set by the loader when they are loaded, read by the products as ready."""

    def __init__(self, n):
        self.loaded, self.turned = [False] * n, [0] * n

    def __setitem__(self, i, value):
        self.loaded[i] = value

    def __getitem__(self, i):
        return self.turned[i] == TURNERS


class Model8(Model):
    def __init__(self, units, stages, slots, **kw):
        super().__init__(units, stages, **kw)
        self.slots = slots
        self.q_full = Queries(len(units))
        self.loaded = [0] * stages           # fillings of a stage that have arrived, not turned yet
        self.raw = [None] * stages
        self.turning = [0] * stages          # warps that have turned their part of the present filling
        self.scale = [None] * slots          # the key tile whose scales are there
        self.scale_full = [0] * slots
        self.key_tiles = 0
        self.scales_flying = []

    def load(self, tile):
        yield from super().load(tile)
        if tile[1] == "k":
            slot = self.key_tiles % self.slots
            self.key_tiles += 1
            self.scale[slot] = None          # from here on they are being written
            self.scales_flying.append([random.randint(0, 2 * self.late), slot, tile])

    def arrive(self):
        for f in list(self.flying):
            f[0] -= 1
            if f[0] < 0:
                self.flying.remove(f)
                self.raw[f[1]] = f[2]
                self.loaded[f[1]] += 1
                self.turning[f[1]] = 0
                self.steps += 1
        for f in list(self.scales_flying):
            f[0] -= 1
            if f[0] < 0:
                self.scales_flying.remove(f)
                self.scale[f[1]] = f[2]
                self.scale_full[f[1]] += 1
                self.steps += 1

    def turner(self):
        ring = keys = values = 0
        for i, (wide, n) in enumerate(self.units):
            while not self.q_full.loaded[i]:
                yield
            for _ in range(random.randint(0, self.delay)):
                yield
            self.q_full.turned[i] += 1
            self.steps += 1
            for _ in range(2 * n):
                stage, turn = ring % self.stages, ring // self.stages
                ring += 1
                while self.loaded[stage] & 1 == turn & 1:
                    yield
                tile = self.raw[stage]
                if tile[1] == "k":
                    slot, times = keys % self.slots, keys // self.slots
                    keys += 1
                    while self.scale_full[slot] & 1 == times & 1:
                        yield
                else:
                    slot = values % self.slots
                    values += 1
                want = (tile[0], "k", tile[2])
                for _ in range(random.randint(0, self.delay)):
                    if self.scale[slot] != want:
                        raise Wrong(("scales", self.scale[slot], want))
                    yield
                if self.scale[slot] != want:
                    raise Wrong(("scales", self.scale[slot], want))
                if self.raw[stage] != tile:
                    raise Wrong("filled while it is turned")
                self.turning[stage] += 1
                self.steps += 1
                if self.turning[stage] == TURNERS:
                    self.content[stage] = tile
                    self.filled[stage] += 1

    def run(self):
        procs = [self.loader(), self.products(0), self.products(1), self.softmax(0), self.softmax(1)]
        procs += [self.turner() for _ in range(TURNERS)]
        idle, before = 0, None
        while procs:
            self.arrive()
            random.shuffle(procs)
            for p in list(procs):
                try:
                    next(p)
                except StopIteration:
                    procs.remove(p)
            after = (self.loads, len(self.scores[0]), len(self.scores[1]), tuple(self.ready), len(self.outs[0]),
                     len(self.outs[1]), self.steps, tuple(self.met), len(procs))
            idle = idle + 1 if before == after and not self.flying and not self.scales_flying else 0
            before = after
            if idle > 10 + 8 * self.delay:
                return False
        return True


@pytest.mark.parametrize("stages, slots", [(5, 4), (10, 8)])  # heads of 128 and 64
def test_every_sequence_of_units_ends(stages, slots):
    rng = random.Random(stages)
    random.seed(stages)
    for trial in range(1200):
        units = random_units(rng)
        assert Model8(units, stages, slots, delay=trial % 5, late=(0, 3, 30)[trial % 3]).run(), units


def test_model_finds_scales_that_are_overwritten():
    """With fewer slots the loads run ahead of what is still to be turned."""
    random.seed(3)
    wrong = 0
    for _ in range(200):
        try:
            wrong += not Model8([(False, 11)] * 4, 5, 2, delay=4, late=3).run()
        except Wrong:
            wrong += 1
    assert wrong > 0


def test_model_finds_a_deadlock():
    random.seed(1)
    assert not Model8([(False, 3), (False, 3)], 1, 4).run()
    assert Model8([(False, 3), (False, 3)], 5, 4).run()
