"""A CPU model of who reads the scales of a cache in 8 bits in the tensor-core kernel
(csrc/gdn_attn_tc.cu): the loader's copies bring a key tile's and its values' into a slot, one of the warps
that turn tiles waits for them, and the softmax reads them between a tile's scores and its weights.  The
rest of the protocol is that of tests/test_cache8_protocol_model.py."""
from __future__ import annotations

import random

import pytest

from tests.test_attn_protocol_model import Wrong, random_units
from tests.test_cache8_protocol_model import Model8


class Scales(Model8):
    def __init__(self, units, stages, slots, **kw):
        super().__init__(units, stages, slots, **kw)
        self.turners = 0
        self.turned_scales = [None] * slots  # the key tile whose scales the softmax may read

    def turner(self):
        first = self.turners == 0
        self.turners += 1
        ring = keys = 0
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
                if first and tile[1] == "k":
                    slot, times = keys % self.slots, keys // self.slots
                    keys += 1
                    while self.scale_full[slot] & 1 == times & 1:
                        yield
                    if self.scale[slot] != tile:
                        raise Wrong(("scales", self.scale[slot], tile))
                    self.turned_scales[slot] = tile
                for _ in range(random.randint(0, self.delay)):
                    yield
                if self.raw[stage] != tile:
                    raise Wrong("filled while it is turned")
                self.turning[stage] += 1
                self.steps += 1
                if self.turning[stage] == 4:
                    self.content[stage] = tile
                    self.filled[stage] += 1

    def softmax(self, x):
        seen = before = 0
        for i, (wide, n) in enumerate(self.units):
            tiles = range(n) if wide else range(x, n, 2)
            for t in tiles:
                while len(self.scores[x]) <= seen:
                    yield
                for stage in self.scores[x][seen][2]:
                    self.hand_back(stage, 1 if wide else 2)
                slot, want = (before + t) % self.slots, (i, "k", t)
                for _ in range(random.randint(0, self.delay) + 1):
                    if self.scale[slot] != want or self.turned_scales[slot] != want:
                        raise Wrong(("scales", self.scale[slot], self.turned_scales[slot], want))
                    yield
                seen += 1
                self.ready[x] += 1
            before += n
            while tiles and i not in self.outs[x]:
                yield
            if not wide and n > 1:
                self.met[x] += 1
                while self.met[x ^ 1] < self.met[x]:
                    yield


@pytest.mark.parametrize("stages, slots", [(5, 4), (10, 8)])  # heads of 128 and 64
def test_every_tile_has_its_own_scales(stages, slots):
    rng = random.Random(stages)
    random.seed(stages)
    for trial in range(1200):
        units = random_units(rng)
        assert Scales(units, stages, slots, delay=trial % 5, late=(0, 3, 30)[trial % 3]).run(), units


def test_model_finds_scales_that_are_overwritten():
    random.seed(3)
    wrong = 0
    for _ in range(200):
        try:
            wrong += not Scales([(False, 11)] * 4, 5, 2, delay=4, late=3).run()
        except Wrong:
            wrong += 1
    assert wrong > 0
