"""A CPU model of what the bf16 attention kernel (csrc/gdn_attn_tc.cu) does once a wait has given
up: a copy or a product's completion is lost, some wait runs out of its time, and from then on every
wait that is not over returns at once.  All roles must come to their end; until then no barrier
outside the kernel's own may be arrived on (the hand-back of stages reads their numbers from shared
memory), and no place may be filled while an earlier copy into it is on its way (its barrier would
be asked for two fillings in one phase)."""
from __future__ import annotations

import random

import pytest


class Wrong(Exception):
    pass


class Barrier:
    """Phase, arrivals and bytes still to come, as the hardware's; told apart by parity only."""

    def __init__(self, count):
        self.count, self.pending, self.bytes, self.phase = count, count, 0, 0

    def arrive(self, expect=0):
        if self.pending == 0:
            raise Wrong("an arrival more than the phase has, while a copy is on its way")
        self.bytes += expect
        self.pending -= 1
        self.turn()

    def landed(self, n):
        self.bytes -= n
        self.turn()

    def turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.pending, self.phase = self.count, self.phase ^ 1

    def over(self, parity):
        return self.phase != parity


def last_values(wide, n):
    """Which X reads each of a unit's last value tiles (None: both), in the order they are loaded:
    before the next unit's first keys, and behind them."""
    if wide:
        return [None], []
    if n == 1:
        return [0], []
    return ([0], [1]) if (n - 1) & 1 else ([1, 0], [])


class Kernel:
    """Units are (wide, tiles).  ``lost``: which of the copies and commits, counted from the start,
    never completes.  ``keep``: no place is handed back any more once a wait has given up; ``stop``:
    the loader loads nothing behind a wait of its own that gave up."""

    def __init__(self, units, stages, lost, keep=True, stop=True):
        self.units, self.stages, self.lost, self.keep, self.stop = units, stages, lost, keep, stop
        self.events, self.abort, self.flying = 0, False, []
        self.full = [Barrier(1) for _ in range(stages)]
        self.empty = [Barrier(2) for _ in range(stages)]
        self.q_full, self.q_empty = Barrier(1), Barrier(2)
        self.s_full = [Barrier(2), Barrier(2)]
        self.ready = [Barrier(1), Barrier(1)]  # all softmax warps of an X as one
        self.o_full = [Barrier(1), Barrier(1)]
        self.used = [None, None]  # stages that the scores of each X free

    def later(self, barrier, nbytes):
        """A copy's bytes or a commit, some steps later or never."""
        if self.events != self.lost:
            self.flying.append([random.randint(0, 6), barrier, nbytes])
        self.events += 1

    def wait(self, barrier, parity):
        """True: over; False: gave up."""
        while not barrier.over(parity):
            if self.abort:
                return False
            yield
        return True

    def loader(self):
        at, turn, q_parity, lost = 0, 0, 1, False

        def load():
            nonlocal at, turn, lost
            if not (yield from self.wait(self.empty[at], turn ^ 1)):
                lost = self.stop
            if not lost:
                self.full[at].arrive(expect=1)
                self.later(self.full[at], 1)
            at += 1
            if at == self.stages:
                at, turn = 0, turn ^ 1

        before, behind = [], []
        for wide, n in self.units:
            for _ in before:
                yield from load()
            if not (yield from self.wait(self.q_empty, q_parity)):
                lost = self.stop
            q_parity ^= 1
            if not lost:
                self.q_full.arrive(expect=1)
                self.later(self.q_full, 1)
            yield from load()
            for _ in behind:
                yield from load()
            for _ in range(2 * (n - 1) if wide else (n > 1) + 2 * max(n - 2, 0)):
                yield from load()
            before, behind = last_values(wide, n)
        for _ in before + behind:
            yield from load()

    # One X's products: every tile of the ring in order (it waits for the other X's too).
    def products(self, x):
        at, turn, q_parity, parity = 0, 0, 0, 0

        def tile():
            nonlocal at, turn
            stage = at
            yield from self.wait(self.full[stage], turn)
            at += 1
            if at == self.stages:
                at, turn = 0, turn ^ 1
            return stage

        def scores(k, v):
            self.later(self.s_full[x], None)
            self.used[x] = (k, v)
            self.s_full[x].arrive()

        def output():
            nonlocal parity
            yield from self.wait(self.ready[x], parity)
            parity ^= 1

        def last(v, twice):
            yield from output()
            if not (self.abort and self.keep):
                for _ in range(2 if twice else 1):
                    self.later(self.empty[v], None)
            self.later(self.o_full[x], None)

        before, behind = [], []
        for wide, n in self.units + [(None, 0)]:
            for who in before if wide is not None else before + behind:
                v = yield from tile()
                if who is None or who == x:
                    yield from last(v, who is not None)
            if wide is None:
                return
            k = yield from tile()
            yield from self.wait(self.q_full, q_parity)
            q_parity ^= 1
            if x == 0:
                scores(k, -1)
            for who in behind:
                v = yield from tile()
                if who == x:
                    yield from last(v, True)
            if wide:
                if x == 1:
                    scores(k, -1)
                for _ in range(n - 1):
                    v = yield from tile()
                    k = yield from tile()
                    yield from output()
                    scores(k, v)
            else:
                if n > 1:
                    k = yield from tile()
                    if x == 1:
                        scores(k, -1)
                for t in range(2, n):
                    v = yield from tile()
                    k = yield from tile()
                    if t & 1 == x:
                        yield from output()
                        scores(k, v)
            before, behind = last_values(wide, n)
            if self.abort and self.keep:
                pass
            elif x == 0 or wide or n > 1:
                self.later(self.q_empty, None)
            else:
                self.q_empty.arrive()

    def softmax(self, x):
        parity, o_parity = 0, 0
        for wide, n in self.units:
            tiles = range(n) if wide else range(x, n, 2)
            for _ in tiles:
                yield from self.wait(self.s_full[x], parity)
                parity ^= 1
                if not (self.abort and self.keep):
                    if self.used[x] is None:
                        raise Wrong("a barrier from what was never written")
                    for stage in self.used[x]:
                        for _ in range(0 if stage < 0 else 1 if wide else 2):
                            self.empty[stage].arrive()
                yield
                self.ready[x].arrive()
            if tiles:
                yield from self.wait(self.o_full[x], o_parity)
                o_parity ^= 1

    def run(self):
        """False: a role did not come to its end."""
        roles = [self.loader(), self.products(0), self.products(1), self.softmax(0), self.softmax(1)]
        quiet = 0
        for _ in range(20000):
            for f in list(self.flying):
                f[0] -= 1
                if f[0] < 0:
                    self.flying.remove(f)
                    f[1].arrive() if f[2] is None else f[1].landed(f[2])
            random.shuffle(roles)
            before = (len(roles), self.events, self.state())
            for r in list(roles):
                try:
                    next(r)
                except StopIteration:
                    roles.remove(r)
            if not roles:
                return True
            quiet = quiet + 1 if before == (len(roles), self.events, self.state()) and not self.flying else 0
            if quiet > 20:  # a wait's time is over
                if self.abort:
                    return False
                self.abort = True
        return False

    def state(self):
        every = self.full + self.empty + [self.q_full, self.q_empty] + self.s_full + self.ready + self.o_full
        return tuple((b.phase, b.pending, b.bytes) for b in every)


def random_units(rng):
    return [(rng.random() < 0.4, rng.choice((1, 1, 2, 3, 4, 5, 7, 11))) for _ in range(rng.randint(1, 5))]


@pytest.mark.parametrize("stages", [5, 10])
def test_nothing_lost(stages):
    rng = random.Random(stages)
    random.seed(stages)
    for _ in range(300):
        k = Kernel(random_units(rng), stages, lost=-1)
        assert k.run() and not k.abort and all(f[2] is None for f in k.flying)  # no copy is left


@pytest.mark.parametrize("stages", [5, 10])
def test_every_loss_ends_in_bounds(stages):
    rng = random.Random(stages + 1)
    random.seed(stages + 1)
    ends = gave_up = 0
    for _ in range(60):
        units = random_units(rng)
        whole = Kernel(units, stages, lost=-1)
        assert whole.run()
        for lost in range(whole.events):
            k = Kernel(units, stages, lost)
            assert k.run(), (units, lost)
            ends += 1
            gave_up += k.abort
    assert gave_up > ends / 2  # nobody waits for the last commits of a stage


@pytest.mark.parametrize("kw, message", [
    (dict(keep=False, stop=False), "never written"), (dict(keep=False), "on its way"), (dict(stop=False), "on its way")])
def test_model_finds_what_was_mended(kw, message):
    random.seed(3)
    found = 0
    for lost in range(40):
        for units in ([(False, 5)] * 3, [(True, 6), (False, 2), (True, 3)]):
            try:
                Kernel(units, 5, lost, **kw).run()
            except Wrong as e:
                found += message in str(e)
    assert found > 0
