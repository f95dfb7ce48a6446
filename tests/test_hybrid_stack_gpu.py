"""Gated-delta and attention layers together (examples/hybrid_stack.py): a packed prefill, a
prompt's next chunk and single tokens give what one pass over everything gives.

Tolerance.  The two ways differ in how they sum and, in bf16, in what they round: every tensor
between two operations carries a rounding of root mean square at most 2^-8 / sqrt(3) = 2.3e-3 of
its values.  A layer has about ten such roundings in a row, each way has its own, so a layer's
output differs by about sqrt(20) * 2.3e-3 = 1.0e-2 of itself; layers add to a stream of at least
their size with independent errors, so the stream differs by less than twice that.  In fp32 the
same count holds with roundings of 2^-24 and sums of a few hundred terms (2^-24 sqrt(256)), about
1e-6 each: sqrt(20) * 2e-6 = 1e-5, and 1e-4 leaves room for the chunked form's triangular inverse.
"""
from __future__ import annotations

import pytest
import torch

from examples.hybrid_stack import WIDTH, Stack, packed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, tol", [(torch.bfloat16, 2e-2), (torch.float32, 1e-4)], ids=str)
@pytest.mark.parametrize("layers", ["A", "GA", "GGAGA"])
def test_pieces_equal_one_pass(layers, dtype, tol):
    prompts, chunk, steps = [65, 1, 130, 20], 37, 5
    gen = torch.Generator().manual_seed(len(layers))
    tokens = [torch.randn((n + chunk + steps, WIDTH), generator=gen).cuda().to(dtype) for n in prompts]
    stack = Stack(layers, dtype)
    stack.allocate(len(prompts), max(map(len, tokens)))
    got = [list(stack.run(*packed([t[:n] for t, n in zip(tokens, prompts)]), whole=True)[0].split(prompts))]
    part = packed([t[n:n + chunk] for t, n in zip(tokens, prompts)])
    got.append(list(stack.run(*part)[0].split(chunk)))
    for i in range(chunk, chunk + steps):
        x = torch.stack([t[n + i] for t, n in zip(tokens, prompts)])[:, None]
        got.append(list(stack.run(x)))
    pieces = [torch.cat(p) for p in zip(*got)]
    again = Stack(layers, dtype)
    again.allocate(len(prompts), max(map(len, tokens)))
    whole = again.run(*packed(tokens), whole=True)[0].split([len(t) for t in tokens])
    torch.cuda.synchronize()
    for a, b in zip(pieces, whole):
        assert torch.isfinite(a).all()
        a, b = a.double(), b.double()
        assert (a - b).norm() <= tol * b.norm(), float((a - b).norm() / b.norm())
    assert torch.equal(stack.lens, again.lens)
