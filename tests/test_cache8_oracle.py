"""The plain forms in oracle/cache8.py against what they stand for, without a GPU: every e4m3 code
against PyTorch's type, rounding at ties, scales, positions, copies."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn
from oracle import cache8


def test_every_code_is_the_types_value():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache8.DECODE, want, equal_nan=True)
    fine = ~np.isnan(want)
    assert np.array_equal(cache8.encode(want)[fine], codes.numpy()[fine])


def test_rounding_is_to_the_nearest_and_ties_to_even():
    v = np.sort(np.unique(cache8.DECODE[:127]))
    mid = (v[:-1] + v[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, v[:-1], v[1:])
    assert np.array_equal(cache8.decode(cache8.encode(mid)), even)
    assert np.array_equal(cache8.decode(cache8.encode(np.nextafter(mid, 1e9))), v[1:])
    assert np.array_equal(cache8.decode(cache8.encode(np.nextafter(mid, 0))), v[:-1])
    x = torch.randn(4000, dtype=torch.float32, generator=torch.Generator().manual_seed(0)) * 60
    x = x.clamp(-448, 448)
    assert np.array_equal(cache8.encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("top, e", [(0.0, -117), (1e-45, -117), (448.0, 0), (448.1, 1), (896.0, 1), (1.0, -8),
                                    (1.75, -8), (1.7500001, -7), (3.38e38, 120)])
def test_scale_of_a_block(top, e):
    assert cache8.need(top) == 2.0 ** e


def test_far_angles():
    assert abs(float(cache8.PI) - math.pi) < 1e-15
    f = np.float32(0.7123)
    for p in (0, 1, -3, 12345):
        assert abs(math.cos(cache8.angle(p, f)) - math.cos(p * float(f))) < 1e-11
    # whole turns fall away exactly: the angle of p + q is the sum of theirs
    a, b, c = (cache8.angle(p, f) for p in (2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1))
    assert abs(math.remainder(a - b - c, 2 * math.pi)) < 1e-14


def test_copies_read_what_was_there():
    x = np.arange(8.0)
    assert list(cache8.copy_pages(x, [0, 1, 2, 5], [3, 3, 4, 6])) == [0, 1, 2, 3, 2, 5, 5, 7]
    assert list(cache8.copy_pages(x, [0, 3, 9, 2], [3, 5, 1, 2])) == [0, 1, 2, 3, 4, 3, 6, 7]


def test_frequencies():
    f = gdn.rope_inv_freq(64, 10000.0)
    assert f.dtype == torch.float32 and torch.equal(f, (10000.0 ** (-torch.arange(0, 64, 2).double() / 64)).float())
    assert torch.equal(gdn.rope_inv_freq(64, 10000.0, stretch=4.0), (10000.0 ** (-torch.arange(0, 64, 2).double() / 64) / 4).float())
    g = gdn.rope_inv_freq(64, 10000.0, stretch=8.0, trained=4096)
    turns = 4096 * f.double() / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and torch.equal(g[turns <= 1], (f.double() / 8).float()[turns <= 1])
    assert ((g <= f) & (g.double() >= f.double() / 8 * (1 - 1e-6))).all() and (g.diff() < 0).all()
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, stretch=0.5), dict(rot=8, base=-1.0), dict(rot=8, fast=1.0)):
        with pytest.raises(ValueError):
            gdn.rope_inv_freq(**bad)
