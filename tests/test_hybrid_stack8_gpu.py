"""Gated-delta and attention layers together with rotary positions and an 8-bit cache
(examples/hybrid_stack.py): pieces against one pass, and sequences that fork.

Tolerance.  With positions the two ways differ by two more roundings for q and k, which the count
of tests/test_hybrid_stack_gpu.py (ten roundings for a layer and way) has room for: 2e-2.
With a cache in 8 bits both ways round each key and value to e4m3, but not to the same values:
what a block's rows are rounded to depends on the scale that the block had when they were
written, and inputs that differ by a rounding of bf16 may fall on either side of a border, half a
step of e4m3 (2^-4 of the value) apart at the most, as often as the difference is of a step: a
relative difference of e between inputs leaves one of about sqrt(e 2^-4) between their roundings
(a share e / 2^-3 of the values moves by 2^-3), 1.1e-2 for e = 2^-9.  An average over n keys with
like weights shrinks by sqrt(n) what does not fall together, and the largest effect is on rows that see
one key only: a layer's output is off by at most 1.1e-2 sqrt(2) of itself, from keys and values, beside
1.0e-2 from its other roundings, and two of those layers add to a stream of their own size, so that
below 4e-2 is left for the whole.
"""
from __future__ import annotations

import pytest
import torch

from examples.hybrid_stack import WIDTH, Stack, packed

pytestmark = pytest.mark.gpu


def run_pieces(stack, tokens, prompts, chunk, steps):
    got = [list(stack.run(*packed([t[:n] for t, n in zip(tokens, prompts)]), whole=True)[0].split(prompts))]
    part = packed([t[n:n + chunk] for t, n in zip(tokens, prompts)])
    got.append(list(stack.run(*part)[0].split(chunk)))
    for i in range(chunk, chunk + steps):
        got.append(list(stack.run(torch.stack([t[n + i] for t, n in zip(tokens, prompts)])[:, None])))
    return [torch.cat(p) for p in zip(*got)]


@pytest.mark.parametrize("cache8, tol", [(False, 2e-2), (True, 4e-2)])
@pytest.mark.parametrize("layers, rot", [("A", 64), ("GA", 32), ("GAGA", 64)])
def test_pieces_equal_one_pass(layers, rot, cache8, tol):
    prompts, chunk, steps = [65, 1, 130, 20], 37, 5
    gen = torch.Generator().manual_seed(len(layers))
    tokens = [torch.randn((n + chunk + steps, WIDTH), generator=gen).cuda().bfloat16() for n in prompts]
    stacks = [Stack(layers, rot=rot, cache8=cache8) for _ in range(2)]
    for s in stacks:
        s.allocate(len(prompts), max(map(len, tokens)))
    pieces = run_pieces(stacks[0], tokens, prompts, chunk, steps)
    whole = stacks[1].run(*packed(tokens), whole=True)[0].split([len(t) for t in tokens])
    torch.cuda.synchronize()
    for a, b in zip(pieces, whole):
        assert torch.isfinite(a).all()
        a, b = a.double(), b.double()
        assert (a - b).norm() <= tol * b.norm(), float((a - b).norm() / b.norm())


def test_positions_matter():
    """With positions a layer tells the same tokens in another order apart; without, its last row
    does not (to rounding)."""
    tokens = torch.randn((40, WIDTH), generator=torch.Generator().manual_seed(3)).cuda().bfloat16()
    mixed = torch.cat([tokens[:39].flip(0), tokens[39:]])
    for rot in (0, 64):
        last = []
        for t in (tokens, mixed):
            s = Stack("A", rot=rot)
            s.allocate(1, 64)
            last.append(s.run(*packed([t]), whole=True)[0, -1].double())
        off = float((last[0] - last[1]).norm() / last[0].norm())
        assert off < 2e-2 if rot == 0 else off > 2e-2, (rot, off)


@pytest.mark.parametrize("cache8", [False, True])
@pytest.mark.parametrize("held", [47, 48, 5])
def test_fork(cache8, held):
    """A sequence forks in the middle (or at the end) of a page: both go on as if each had been
    alone from the start, bit for bit, though they share their full pages."""
    gen = torch.Generator().manual_seed(held)
    base = torch.randn((held, WIDTH), generator=gen).cuda().bfloat16()
    more = [torch.randn((20, WIDTH), generator=gen).cuda().bfloat16() for _ in range(2)]
    forked = Stack("GA", rot=64, cache8=cache8)
    forked.allocate(2, 80)
    forked.run(*packed([base, base[:1]]), whole=True)  # the second sequence is about to be replaced
    forked.fork(0, 1)
    alone = Stack("GA", rot=64, cache8=cache8)
    alone.allocate(2, 80)
    alone.run(*packed([base, base]), whole=True)
    for i in range(20):
        x = torch.stack([m[i] for m in more])[:, None]
        assert torch.equal(forked.run(x), alone.run(x)), i
    assert torch.equal(forked.lens, alone.lens)
    full = held // 16
    assert torch.equal(forked.table[0, :full], forked.table[1, :full]) and forked.table[0, full] != forked.table[1, full]
