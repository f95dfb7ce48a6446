"""GPU parity of rotary positions against oracle/cache8.py.

Tolerances.  Angles are exact to 2^-29 (2^-32 of a turn) and taken to fp32 as quarter turns and a rest of at most
pi / 4, off by 2^-25 of it; sine and cosine are off by at most 2 units of 2^-24; so a turned
element a cos - b sin, with its two products and one sum in fp32, is off by at most
mscale (|a| + |b|) 2^-24 (2 + 1 + 1 + 1 + pi / 4) < 6 2^-24 mscale (|a| + |b|), and its rounding to
bf16 adds 2^-8 of the result.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn
from oracle import cache8

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, x, pos, freq, interleaved, mscale, backward=False):
    x64 = f64(x).reshape(-1, *x.shape[2:])
    want = cache8.rope(x64, pos, freq.numpy(), interleaved, mscale, backward)
    mag, half = np.abs(x64), len(freq)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    bound = np.zeros_like(mag)
    bound[..., a] = bound[..., b] = 6 * 2.0 ** -24 * abs(mscale) * (mag[..., a] + mag[..., b])
    if x.dtype == torch.bfloat16:
        bound[..., :2 * half] += 2.0 ** -8 * (np.abs(want[..., :2 * half]) + bound[..., :2 * half])
    err = np.abs(f64(got).reshape(want.shape) - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


def positions(q_lens, kv_lens=None):
    kv_lens = q_lens if kv_lens is None else kv_lens
    return [p for a, b in zip(q_lens, kv_lens) for p in range(b - a, b)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d, rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 112)])
def test_packed(dtype, interleaved, d, rot):
    dt, q_lens, kv = DTYPES[dtype], [1, 0, 7, 40, 1], [1000, 5, 7, 99, 1]
    q, k = normal((1, 49, 6, d), dt, 1), normal((1, 49, 2, d), dt, 2)
    freq = gdn.rope_inv_freq(rot, 10000.0)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32).cuda()
    lens, flags = torch.tensor(kv, dtype=torch.int32).cuda(), torch.full((1,), 3, dtype=torch.int32, device="cuda")
    for back, entry in ((False, gdn.gdn_rope_fwd), (True, gdn.gdn_rope_bwd)):
        qo, ko = entry(q.cuda(), k.cuda(), freq.cuda(), interleaved=interleaved, mscale=1.25, kv_lens=lens, cu_seqlens=cu, flags=flags)
        assert gdn.gdn_read_device_flags(flags) == 0
        for got, x in ((qo, q), (ko, k)):
            check(got, x, positions(q_lens, kv), freq, interleaved, 1.25, back)
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("B, T, H, HKV", [(1, 1, 1, 1), (5, 1, 32, 8), (2, 33, 3, 5), (1, 5001, 1, 1)])
def test_batch(dtype, B, T, H, HKV):
    dt, d = DTYPES[dtype], 64
    q, k = normal((B, T, H, d), dt, 1), normal((B, T, HKV, d), dt, 2)
    freq = gdn.rope_inv_freq(16, 500000.0, stretch=4.0, trained=4096)
    qo, ko = gdn.gdn_rope_fwd(q.cuda(), k.cuda(), freq.cuda())
    pos = positions([T] * B)
    check(qo, q, pos, freq, False, 1.0)
    check(ko, k, pos, freq, False, 1.0)
    only, none = gdn.gdn_rope_fwd(q.cuda(), None, freq.cuda())
    assert none is None and torch.equal(only, qo)


def test_far_positions_and_odd_frequencies():
    """Any 32-bit position, before the first one too; frequencies of every size and sign, zero and
    the smallest among them."""
    lens = [131072, 1 << 24, (1 << 24) + 1, 2 ** 31 - 1025, 0, 1]
    freq = torch.tensor([1.0, 0.7123, 6.2831855, 100.3, 1e6, -0.3, 0.0, 1e-45, 2.0 ** -20, 2.0 ** 62, 1e-4, 3e-30, 0.5, 1.0, 0.1, 12.9898])
    x = normal((len(lens), 3, 2, 64), torch.float32, 4)
    q, _ = gdn.gdn_rope_fwd(x.cuda(), None, freq.cuda(), kv_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    check(q, x, positions([3] * len(lens), lens), freq, False, 1.0)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
def test_slices_in_place(dtype, interleaved):
    """q and k of one projection's output turned where they lie; the values between stay."""
    dt, B, T, H, HKV, d = DTYPES[dtype], 2, 37, 4, 2, 64
    x = normal((B, T, H + 2 * HKV + 1, d), dt, 11)
    freq = gdn.rope_inv_freq(32)
    y = x.cuda()
    q, k = y[:, :, :H], y[:, :, H + 1:H + 1 + HKV]
    want = gdn.gdn_rope_fwd(q, k, freq.cuda(), interleaved=interleaved)
    check(want[0], x[:, :, :H], positions([T] * B), freq, interleaved, 1.0)
    gdn.gdn_rope_fwd(q, k, freq.cuda(), interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    rest = [H] + list(range(H + 1 + HKV, H + 2 * HKV + 1))
    assert torch.equal(y[:, :, rest].cpu(), x[:, :, rest])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(interleaved):
    """The gradient of sum(c * rope(x)) by the formula is rope_bwd(c); against differences too:
    the operator is linear, so a difference over any step has no error but rounding."""
    x, c = normal((1, 50, 4, 64), torch.float32, 1), normal((1, 50, 4, 64), torch.float32, 2)
    freq = gdn.rope_inv_freq(48)
    kw = dict(interleaved=interleaved, mscale=1.3)

    def loss(y):
        return float((gdn.gdn_rope_fwd(y.cuda(), None, freq.cuda(), **kw)[0].double().cpu() * c.double()).sum())

    grad, _ = gdn.gdn_rope_bwd(c.cuda(), None, freq.cuda(), **kw)
    check(grad, c, positions([50]), freq, interleaved, 1.3, True)
    gen = torch.Generator().manual_seed(5)
    for _ in range(8):
        way = torch.randn(x.shape, generator=gen)
        # 12800 outputs, each off by at most 6 2^-24 1.3 (|a| + |b|) for inputs of up to 10
        slack = 2 * float((6 * 2.0 ** -24 * 1.3 * 20 * c.abs().double()).sum())
        assert abs(loss(x + way) - loss(x - way) - 2 * float((grad.double().cpu() * way.double()).sum())) <= slack
    # back and forth: the transpose of a rotation undoes it but for mscale^2
    back = gdn.gdn_rope_bwd(gdn.gdn_rope_fwd(x.cuda(), None, freq.cuda(), **kw)[0], None, freq.cuda(), **kw)[0].cpu()
    assert torch.allclose(back[..., :48], 1.69 * x[..., :48], rtol=0, atol=20 * 6 * 2.0 ** -24 * 1.69 * 2)


def test_malformed_lengths():
    x = normal((1, 30, 2, 64), torch.bfloat16, 1).cuda()
    freq = gdn.rope_inv_freq(64, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    good, _ = gdn.gdn_rope_fwd(x, None, freq, cu_seqlens=torch.tensor([0, 10, 20, 30], dtype=torch.int32).cuda(), flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0
    for cu, lens, kept in (([0, 10, 20, 30], [10, -3, 10], [*range(10), *range(20, 30)]), ([0, 10, 40, 30], [10, 10, 10], range(10)),
                           ([5, 10, 20, 30], [5, 10, 10], range(10, 30)), ([0, 10, 20, 25], [10, 10, 5], range(20))):
        out = torch.full_like(x, 9.0)
        gdn.gdn_rope_fwd(x, None, freq, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), q_out=out, flags=flags,
                         kv_lens=torch.tensor(lens, dtype=torch.int32).cuda())
        assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS, cu
        kept = list(kept)
        assert torch.equal(out[:, kept], good[:, kept])


def test_streams_and_graphs():
    q, k = normal((64, 1, 8, 128), torch.bfloat16, 1).cuda(), normal((64, 1, 2, 128), torch.bfloat16, 2).cuda()
    freq, lens = gdn.rope_inv_freq(128, device="cuda"), torch.arange(1, 65, dtype=torch.int32).cuda()
    want = gdn.gdn_rope_fwd(q, k, freq, kv_lens=lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = gdn.gdn_rope_fwd(q, k, freq, kv_lens=lens, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.gdn_rope_fwd(q, k, freq, kv_lens=lens)
    lens += 1000
    graph.replay()
    again = gdn.gdn_rope_fwd(q, k, freq, kv_lens=lens)
    torch.cuda.synchronize()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1]) and not torch.equal(out[0], want[0])
