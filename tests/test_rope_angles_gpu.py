"""The angles of rotary positions by themselves: pairs (1, 0) in fp32 become (cos, sin).

Bound.  An angle is off by at most 2^-25; the functions' results by one unit in the last place, 2^-24 at the most; times
mscale = 1 and with products of 1 and 0 nothing is added: 2^-24 + 2^-25.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn
from oracle import cache8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("last", [400, 131072, (1 << 31) - 1])
def test_sine_and_cosine(last, interleaved):
    T, d = 400, 128
    freq = gdn.rope_inv_freq(d)
    x = torch.zeros((1, T, 1, d), device="cuda")
    x[..., 0::2] = 1
    if not interleaved:
        x = torch.cat([torch.ones((1, T, 1, d // 2)), torch.zeros((1, T, 1, d // 2))], -1).cuda()
    lens = torch.tensor([last], dtype=torch.int32, device="cuda")
    y, _ = gdn.gdn_rope_fwd(x, None, freq.cuda(), interleaved=interleaved, kv_lens=lens)
    y = y[0, :, 0].double().cpu().numpy()
    c, s = (y[:, 0::2], y[:, 1::2]) if interleaved else (y[:, :d // 2], y[:, d // 2:])
    want = np.array([[cache8.angle(last - T + t, f) for f in freq.tolist()] for t in range(T)])
    bound = 2.0 ** -24 + 2.0 ** -25
    assert np.abs(c - np.cos(want)).max() <= bound and np.abs(s - np.sin(want)).max() <= bound
    assert math.isclose(float(np.abs(c ** 2 + s ** 2 - 1).max()), 0, abs_tol=4 * bound)
