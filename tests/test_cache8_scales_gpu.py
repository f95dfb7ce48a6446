"""Attention over a cache in 8 bits: what the scales of blocks may not do, and how near the outputs are.

Bounds, against 64-bit attention over the dequantised cache, for both kernels.  Of a row, over the keys j that
it sees, with weights w_j (of sum 1), |s|_j = scale sum_i |q_i k_ji|, v_j = b_j c_j (scale and 8-bit value):
A = sum_j w_j |v_j|, E = sum_j w_j |s|_j, P = sum_j w_j |s|_j |v_j|, Z = max_j (w_j b_j) sum_j |c_j|.
* Operands are exact, a score is a sum of 128 products in 32 bits and one or two products with scales: it is off by
  at most 2^-18 |s|_j.  Exponents are taken relative to a maximum of about the log-sum-exp's size:
  |d lse| <= 2^-18 E + 2^-20 |lse| + 1e-6 to first order.
* A weight times its scale is rounded to fp16 (2^-11 of it) once.  Below fp16's normal numbers the step is 2^-24, and
  the largest of them is at least 2^5.5, so a rounding there is at most 2^-30.5 of that; there are up to three where
  a maximum moves (two steps of a factor): 2^-28 Z.
* The output is rounded to bf16 once: 2^-8 |o|, or half the step below its normal numbers, 2^-134.
So |d o| <= 1.01 (2^-11 A + 2^-8 |o|) + 2^-134 + 2^-28 Z + 2^-18 (P + E A) + (2^-20 |lse| + 2^-17) A.  Over many random values
a rounding's root mean square is at most its largest error over sqrt(3): sqrt(2^-16 + 2^-22) / sqrt(3) = 2.28e-3 of
the norm.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import attn
from tests.test_cache8_gpu import device, f64, gdn, paged, room, run  # noqa: F401  (a fixture among them)

pytestmark = pytest.mark.gpu


def key_scales(x, which, n, L):
    """[L, HKV] the scale of each key of sequence n."""
    page, j = x["codes"][which].shape[1], np.arange(L)
    return x["scales"][which][x["table"][n].numpy()[j // page], j % page // 16].astype(np.float64)


def parts(x, q, q_lens, scale, lse):
    """E, P and Z of every row (and element)."""
    Ttot, H, d = q.shape
    E, P, Z, at = np.zeros((Ttot, H)), np.zeros((Ttot, H, d)), np.zeros((Ttot, H, d)), 0
    for n, nq in enumerate(q_lens):
        k, v = x["values"][0][n], x["values"][1][n]
        L, HKV = k.shape[:2]
        b = key_scales(x, 1, n, L)
        codes = np.abs(v) / b[..., None]
        for t in range(nq):
            end = L - nq + t + 1
            if end <= 0:
                continue
            for h in range(HKV):
                hs = slice(h * (H // HKV), (h + 1) * (H // HKV))
                y = q[at + t, hs]
                w = np.exp(scale * (y @ k[:end, h].T) - lse[at + t, hs, None])
                ws = w * (scale * (np.abs(y) @ np.abs(k[:end, h]).T))
                E[at + t, hs], P[at + t, hs] = ws.sum(-1), ws @ np.abs(v[:end, h])
                Z[at + t, hs] = (w * b[:end, h]).max(-1)[:, None] * codes[:end, h].sum(0)
        at += nq
    return E, P, Z


def close(got, x, q_lens, d, rows=None, scale=None, whole=True):
    """rows: token rows that are looked at (all); whole: there are enough random values for a mean."""
    scale = scale or d ** -0.5
    q = f64(x["q"]).reshape(-1, *x["q"].shape[2:])
    ref, ref_lse, A, _ = attn.attention(q, *x["values"], q_lens, scale)
    o, lse = f64(got[0]).reshape(ref.shape), f64(got[1]).reshape(ref_lse.shape)
    E, P, Z = parts(x, q, q_lens, scale, ref_lse)
    if rows is not None:
        o, lse, ref, ref_lse, A, E, P, Z = (y[rows] for y in (o, lse, ref, ref_lse, A, E, P, Z))
    assert np.isfinite(o).all() and np.array_equal(np.isneginf(lse), np.isneginf(ref_lse)) and not np.isnan(lse).any()
    sees = ~np.isneginf(ref_lse)
    of_lse = 2.0 ** -20 * np.where(sees, np.abs(ref_lse), 0)
    worst = np.abs(lse[sees] - ref_lse[sees]) / (2.0 ** -18 * E + of_lse + 1e-6)[sees]
    assert worst.size == 0 or worst.max() <= 1, ("lse", worst.max(), int((worst > 1).sum()))
    bound = (1.01 * (2.0 ** -11 * A + 2.0 ** -8 * np.abs(ref)) + 2.0 ** -134 + 2.0 ** -28 * Z + 2.0 ** -18 * (P + E[..., None] * A)
             + (of_lse[..., None] + 2.0 ** -17) * A)
    worst = np.abs(o - ref) / bound
    assert worst.max() <= 1, ("o", worst.max(), int((worst > 1).sum()))
    if whole:
        assert np.linalg.norm(o - ref) <= 2.28e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens, kv, H, HKV", [
    ([1] * 9, [1, 16, 17, 128, 129, 300, 0, 777, 2000], 16, 2),
    ([40, 1, 130, 5], [300, 41, 130, 1001], 8, 2),
    ([300], [611], 4, 1),
], ids=str)
def test_how_near(room, d, q_lens, kv, H, HKV):  # noqa: F811
    x = paged(q_lens, kv, H, HKV, d, 32, seed=31 + d, spread=3.0)
    close(run(x), x, q_lens, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens", [[1], [64], [200]], ids=str)
def test_scales_that_are_no_powers_of_two_are_exact(room, d, q_lens):  # noqa: F811
    rng = np.random.RandomState(5)

    def change(which, c, s, n):
        return c, (s * rng.uniform(0.5, 2.0, s.shape)).astype(np.float32)

    x = paged(q_lens, [333], 8, 2, d, 16, seed=3, spread=2.0, change=change)
    close(run(x), x, q_lens, d, whole=q_lens != [1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up", [12, 20, 40, 100])
@pytest.mark.parametrize("which_up", [0, 1], ids=["keys", "values"])
@pytest.mark.parametrize("nq, past, start", [(40, 0, 32), (100, 23, 96), (256, 0, 128), (300, 400, 560)])
def test_later_scales_reach_no_earlier_token(room, d, up, which_up, nq, past, start):  # noqa: F811
    """Blocks from position `start` on have much larger keys or values: tokens before it are as near as ever."""
    def change(which, c, s, n):
        if which == which_up:
            s[start // 16:] *= np.float32(2.0 ** up)
        return c, s

    x = paged([nq], [nq + past], 4, 2, d, 16, seed=12, spread=1.0, change=change)
    close(run(x), x, [nq], d, rows=slice(0, start - past), whole=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [1, 64])
@pytest.mark.parametrize("apart", [16, 24, 40, 70])
def test_small_blocks_beside_large_ones_that_weigh_little(room, d, nq, apart):  # noqa: F811
    """Blocks of one tile whose values are 2^apart times their neighbours', with scores so low that the small ones make up
    the output: neighbours' scales take no bits from them.  Their keys are up to 2^11 times as large, too."""
    L, H = 700, 4
    x = paged([nq], [L], H, 2, d, 16, seed=7, spread=0.0, q_std=0.5)
    big = np.arange(-(-L // 16)) % 3 == 1
    x["q"] = x["q"].abs() + 0.5
    for which in range(2):
        values = x["values"][which][0]
        for i in np.flatnonzero(big):
            pg, rows = int(x["table"][0, i]), min(16, L - 16 * i)
            if which == 0:  # all of one sign: scores far below the others
                x["codes"][0][pg, :rows] = 0xe4      # -48
                x["scales"][0][pg] = 2.0 ** min(apart // 2, 11)
                values[16 * i:16 * i + rows] = -48 * 2.0 ** min(apart // 2, 11)
            else:
                x["scales"][1][pg] *= np.float32(2.0 ** apart)
                values[16 * i:16 * i + rows] *= 2.0 ** apart
    close(run(x), x, [nq], d, whole=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [1, 64])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 10, 2.0 ** 25, 2.0 ** 100])
def test_tiles_of_zero_values_keep_their_weight(room, d, nq, size):  # noqa: F811
    """Whole key tiles of zero values (at the smallest scale), the others as large as `size`: every key counts in the
    sum of the weights."""
    def change(which, c, s, n):
        if which:
            s *= np.float32(size)
            c[128:512], s[8:32] = 0, 2.0 ** -117
            c[640:], s[40:] = 0, 2.0 ** -117
        return c, s

    x = paged([nq], [900], 4, 2, d, 64, seed=19, spread=0.0, change=change)
    close(run(x), x, [nq], d, whole=nq > 1)


@pytest.mark.parametrize("H, HKV, n", [(4, 2, 1), (8, 8, 60), (16, 4, 700)], ids=["blocks", "eight heads", "warps"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [1, 2, 8])
def test_large_values_behind_zeros(d, nq, H, HKV, n):
    """A token that has seen zero values alone, or nearly so by its weights, beside keys that it does not see (or that weigh
    nothing) with very large ones: its output is zero (or theirs), not NaN."""
    nq = min(nq, 8 * HKV // H)

    def change(which, c, s, i):
        if which:
            c[:144], s[:9] = 0, 2.0 ** -117
            s[9:] *= np.float32(2.0 ** 20)
        elif nq == 1:  # the last keys weigh 2^-250 and less
            c[:] = 0
            c[144:], s[9:] = 0xe4, 2.0 ** 4
        return c, s

    L = [144 + (nq + 1) // 2 + i % 3 % nq for i in range(n)]
    x = paged([nq] * n, L, H, HKV, d, 16, seed=23, spread=0.0, q_std=0.5, change=change)
    x["q"] = x["q"].abs().reshape(n, nq, H, d) + 0.5
    got = run(x, cu_seqlens=None)
    close(got, x, [nq] * n, d, whole=False)
    blind = 144 - (np.array(L) - nq)  # a sequence's tokens that see zeros alone
    for i in range(n):
        assert (got[0][i, :max(blind[i], 0)] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens", [[1, 1], [64, 200]], ids=str)
@pytest.mark.parametrize("size", [2.0 ** -117, 2.0 ** -126, 1.25 * 2.0 ** -130, 2.0 ** 110])
def test_scales_at_both_ends(room, d, q_lens, size):  # noqa: F811
    """All values' scales near the smallest or largest numbers, also below the normal ones."""
    def change(which, c, s, n):
        if which:
            s[:] = np.float32(size)
        return c, s

    x = paged(q_lens, [300, 700], 4, 2, d, 16, seed=29, spread=0.0, q_std=0.5, change=change)
    close(run(x), x, q_lens, d, whole=False)


@pytest.mark.parametrize("nq", [1, 64])
def test_a_maximum_that_lags_over_the_smallest_values(room, nq):  # noqa: F811
    """The smallest scale of the write, scores that rise by less than what a maximum is let stand."""
    L, d = 512, 64

    def change(which, c, s, n):
        if which:
            s[:] = 2.0 ** -117
        else:  # scores 0, then 7.5 (in powers of two) from the second key tile on
            c[:128], c[128:], s[:] = 0, 0x38, 7.5 * np.log(2) / 8
        return c, s

    x = paged([nq], [L], 4, 2, d, 16, seed=37, spread=0.0, change=change)
    x["q"] = torch.ones_like(x["q"])
    close(run(x), x, [nq], d, whole=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens", [[1, 1], [64, 200]], ids=str)
def test_scores_of_the_largest_size(room, d, q_lens):  # noqa: F811
    """Scores of up to 2^21 in magnitude, over blocks of different sizes."""
    x = paged(q_lens, [300, 700], 4, 2, d, 16, seed=43, spread=2.0)
    q = f64(x["q"])[0]
    top = max(float(np.abs(q[:, 2 * h:2 * h + 2] @ k[:, h].T).max()) for k in x["values"][0] for h in range(2))
    scale = float(np.float32(2.0 ** 21 / top))
    close(run(x, scale=scale), x, q_lens, d, scale=scale, whole=False)
