"""Plain 64-bit forms, in numpy, of the operators around a cache held in 8 bits: e4m3 values, the
quantising write, the copy of pages, rotary positions."""
from __future__ import annotations

from decimal import Decimal, getcontext

import numpy as np

BLOCK = 16  # tokens that share a scale


def _table():
    code = np.arange(256)
    sign, power, part = np.where(code & 128, -1.0, 1.0), (code >> 3) & 15, code & 7
    value = np.where(power == 0, part * 2.0 ** -9, (8 + part) * 2.0 ** (power - 10.0))
    value[(code & 127) == 127] = np.nan
    return sign * value


DECODE = _table()


def decode(codes):
    return DECODE[np.asarray(codes)]


def encode(x):
    """64-bit values to the nearest e4m3 code, ties to even; at most 448, NaN to 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 1e6)
    power = np.maximum(np.where(mag > 0, np.frexp(mag)[1] - 1, -6), -6)  # of the first bit; at least 2^-6
    steps = np.rint(np.ldexp(mag, 3 - power)).astype(np.int64)  # 8..16 of them, or 0..8 at 2^-6
    code = np.minimum((power + 6) * 8 + steps, 126)             # a carry goes on into the exponent
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def need(top):
    """The smallest power of two (2^-117 to 2^120) with top <= 448 times it."""
    e = -117
    while e < 120 and top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, codes, scales, table, kv_lens, q_lens):
    """Write rows x [Ttot, HKV, d] into copies of codes [n_pages, page, HKV, d] uint8 and scales
    [n_pages, page / 16, HKV]; returns them."""
    codes, scales = np.array(codes), np.array(scales)
    page, at = codes.shape[1], 0
    for n, nq in enumerate(q_lens):
        end, past = int(kv_lens[n]), int(kv_lens[n]) - nq
        for lo in range(max(past, 0) // BLOCK * BLOCK, end, BLOCK) if nq else ():
            pg, inside = table[n][lo // page], lo % page
            pos = np.arange(lo, lo + BLOCK)
            new, old = (pos >= past) & (pos < end), pos < past
            rows = np.asarray(x[at + pos[new] - past], dtype=np.float64)
            for h in range(codes.shape[2]):
                block = codes[pg, inside:inside + BLOCK, h]
                r = rows[:, h]
                fine = np.isfinite(r)
                s = need(np.abs(r[fine]).max(initial=0.0))
                if old.any():
                    was = float(scales[pg, inside // BLOCK, h])
                    s = max(s, was)
                    if s > was:
                        # the quotient is taken in 32 bits, and so is its product
                        down = np.float32(was) / np.float32(s)
                        block[old] = encode((decode(block[old]).astype(np.float32) * down).astype(np.float64))
                block[new] = encode(np.where(fine, r, np.nan).astype(np.float32) / np.float32(s))
                scales[pg, inside // BLOCK, h] = s
        at += nq
    return codes, scales


def dequantise(codes, scales):
    """[n_pages, page, HKV, d] 64-bit values."""
    return decode(codes) * np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, 1)[..., None]


def copy_pages(array, src, dst):
    """Pairs that nothing speaks against, from the array as it was."""
    array, out = np.asarray(array), np.array(array)
    pages = range(len(array))
    for i, (s, d) in enumerate(zip(src, dst)):
        others = [p for j, p in enumerate(zip(src, dst)) if j != i]
        if s in pages and d in pages and not any(d in p for p in others):
            out[d] = array[s]
    return out


def _pi():
    getcontext().prec = 60
    a, b, t, p = Decimal(1), 1 / Decimal(2).sqrt(), Decimal("0.25"), Decimal(1)
    for _ in range(8):  # arithmetic-geometric mean: digits double each time
        n = (a + b) / 2
        t -= p * (a - n) ** 2
        a, b, p = n, (a * b).sqrt(), 2 * p
    return (a + b) ** 2 / (4 * t)


PI = _pi()


def angle(pos, freq):
    """pos * freq, both exact, less whole turns: 64 bits for any position."""
    x = Decimal(int(pos)) * Decimal(float(freq))
    turns = (x / (2 * PI)).to_integral_value()
    return float(x - turns * 2 * PI)


def rope(x, pos, inv_freq, interleaved, mscale, backward=False):
    """x [T, heads, d] turned at positions pos [T]; inv_freq float32 [rot / 2]."""
    x = np.asarray(x, dtype=np.float64)
    y, half = np.array(x), len(inv_freq)
    th = np.array([[angle(p, f) for f in inv_freq] for p in pos])[:, None]
    c, s = mscale * np.cos(th), mscale * np.sin(th) * (-1 if backward else 1)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y
