"""Which pages sequences of examples/hybrid_stack.py hold after several forks, on the CPU (at the end of a page, where none
is copied): what a sequence writes next belongs to it alone."""
from __future__ import annotations

import pytest
import torch

from examples.hybrid_stack import PAGE, Stack


def stack(lens):
    s = Stack("A", device="cpu")
    s.allocate(len(lens), 5 * PAGE)
    s.lens += torch.tensor(lens, dtype=torch.int32) * PAGE
    return s


def pages_to_write(s, i):
    return s.table[i, int(s.lens[i]) // PAGE:].tolist()


def check(s):
    for i in range(len(s.lens)):
        others = [p for j in range(len(s.lens)) if j != i for p in s.table[j].tolist()]
        assert not set(pages_to_write(s, i)) & set(others), i


def test_a_child_becomes_another_ones_copy():
    s = stack([3, 0, 1, 0])
    s.fork(0, 1)
    check(s)
    assert s.table[0, :3].equal(s.table[1, :3])
    s.fork(2, 1)  # shorter than what it shared before: its table held the first parent's pages
    check(s)
    assert s.table[2, :1].equal(s.table[1, :1]) and int(s.lens[1]) == PAGE
    s.fork(1, 3)
    check(s)


def test_pages_that_are_shared_are_not_given_up():
    s = stack([3, 0, 1])
    s.fork(0, 1)
    with pytest.raises(ValueError, match="shared"):
        s.fork(2, 0)  # the first child still reads its pages
    with pytest.raises(ValueError, match="shared"):
        s.fork(1, 0)
    with pytest.raises(ValueError):
        s.fork(2, 2)
    check(s)
