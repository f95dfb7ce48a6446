"""GPU parity of the operators around a cache held in 8 bits: attention over it, the quantising
write, the copy of pages.  The write and the copy are compared bit for bit with oracle/cache8.py.

Tolerances of attention, against 64-bit attention over the dequantised cache.  Let
A = sum_j w_j |v_j| (elementwise) and S = max_j scale sum_i |q_i k_ji| over a row's visible keys.
* e4m3 values are exact in fp16 and bf16, a cache's scales (powers of two) in both, and q, scaled
  by a power of two for its row, in fp16 down to 2^-28 of the row's largest element, with an error
  of at most 2^-39 of that below.  So a score is a sum of 128 exact products in fp32, off by at most
  2^-18 S; the log-sum-exp by as much, plus its own rounding:
  |d lse| <= 2^-18 S + 2^-20 |lse| + 1e-6.
* The weights are rounded once for their product with v, to bf16 at the coarsest (2^-8 of each), the
  output once (2^-8): |d o| <= 2^-8 (A + |o|) * 1.01 + (2^-17 S + 2^-17) A, and over a whole result
  the relative Frobenius error stays below sqrt(2) 2^-8 / sqrt(3) = 3.2e-3 (each rounding's root
  mean square is at most 2^-8 / sqrt(3) of its value, evenly spread and of random sign).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn
from oracle import attn, cache8

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def codes_of(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def check(got, q, ks, vs, q_lens, scale, what=""):
    o, lse = got
    ref, ref_lse, A, S = attn.attention(f64(q).reshape(-1, *q.shape[2:]), ks, vs, q_lens, scale)
    o, lse = f64(o).reshape(ref.shape), f64(lse).reshape(ref_lse.shape)
    blind = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), blind), what
    assert (o[blind] == 0).all(), what
    assert np.isfinite(o).all() and np.isfinite(lse[~blind]).all(), what
    d = np.abs(lse[~blind] - ref_lse[~blind])
    bad = d > 2.0 ** -18 * S[~blind] + 2.0 ** -20 * np.abs(ref_lse[~blind]) + 1e-6
    assert not bad.any(), (what, "lse", float(d.max()), int(bad.sum()))
    bound = (2.0 ** -17 * S[..., None] + 2.0 ** -17) * A + 2.0 ** -8 * 1.01 * (A + np.abs(ref))
    rel = np.linalg.norm(o - ref) / max(np.linalg.norm(ref), 1e-300)
    assert rel <= 3.2e-3 or ref.size < 10000, (what, rel)  # a mean needs many values
    d = np.abs(o - ref)
    bad = d > bound
    assert not bad.any(), (what, float((d / np.maximum(bound, 1e-300)).max()), int(bad.sum()))


def quantised(x, spread, rng):
    """Rows x [L, HKV, d] as blocks: (codes, scales, values); blocks differ in size by up to 2^spread."""
    L, HKV, d = x.shape
    blocks = -(-L // 16)
    full = np.zeros((blocks * 16, HKV, d))
    full[:L] = x
    full *= np.repeat(2.0 ** rng.uniform(-spread, spread, (blocks, HKV)), 16, 0)[..., None]
    top = np.abs(full).reshape(blocks, 16, HKV, d).max((1, 3))
    scales = np.array([[cache8.need(t) for t in row] for row in top]).reshape(blocks, HKV).astype(np.float32)
    codes = cache8.encode(full / np.repeat(scales, 16, 0)[..., None].astype(np.float64))
    values = cache8.decode(codes) * np.repeat(scales, 16, 0)[..., None].astype(np.float64)
    return codes, scales, values[:L]


@pytest.fixture(params=[0, 1 << 18], ids=["short table", "long table"])
def room(request):
    """Positions that a table has room for at least.  A call's kernels are chosen by that: with a short
    table all of these calls are small, and the kernel for few rows has chunks too."""
    global _room
    _room = request.param
    yield
    _room = 0


_room = 0


def paged(q_lens, kv_lens, H, HKV, d, page, seed, spare=3, spread=2.0, q_std=2.0, change=None):
    """A cache whose unheld rows are NaN, unheld blocks' scales too, pages in random order, table
    entries past the last page out of range.  change(which, codes, scales, n): of one sequence."""
    rng = np.random.RandomState(seed)
    N = len(kv_lens)
    held = [-(-n // page) for n in kv_lens]
    n_pages, width = sum(held) + spare, max(max(held), 1, _room // page) + 1
    order = rng.permutation(n_pages)
    table = np.full((N, width), 1 << 30, dtype=np.int32)
    x = dict(codes=[], scales=[], values=[])
    for which in range(2):
        codes = np.full((n_pages, page, HKV, d), 0x7f, dtype=np.uint8)
        scales = np.full((n_pages, page // 16, HKV), np.nan, dtype=np.float32)
        values, at = [], 0
        for n in range(N):
            c, s, v = quantised(rng.randn(kv_lens[n], HKV, d), spread[which] if isinstance(spread, tuple) else spread, rng)
            if change:
                c, s = change(which, c, s, n)
                v = (cache8.decode(c) * np.repeat(s, 16, 0)[..., None].astype(np.float64))[:kv_lens[n]]
            values.append(v)
            for i in range(held[n]):
                pg = table[n, i] = order[at + i]
                rows = min((i + 1) * page, kv_lens[n]) - i * page
                codes[pg, :rows] = c[i * page:i * page + rows]
                some = -(-rows // 16)
                scales[pg, :some] = s[i * page // 16:i * page // 16 + some]
            at += held[n]
        x["codes"].append(codes)
        x["scales"].append(scales)
        x["values"].append(values)
    x["q"] = normal((1, sum(q_lens), H, d), torch.bfloat16, seed + 7, q_std)
    x["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)
    x["table"], x["lens"] = torch.tensor(table), torch.tensor(kv_lens, dtype=torch.int32)
    return x


def device(x):
    k, v = (torch.tensor(c).cuda().view(E4M3) for c in x["codes"])
    ks, vs = (torch.tensor(s).cuda() for s in x["scales"])
    return k, v, ks, vs, x["table"].cuda(), x["lens"].cuda()


def run(x, **kw):
    if "cu_seqlens" not in kw:
        kw["cu_seqlens"] = x["cu"].cuda()
    return gdn.gdn_attn_paged_fp8_fwd(x["q"].cuda(), *device(x), **kw)


def check_paged(got, x, q_lens, d, what="", scale=None):
    check(got, x["q"], *x["values"], q_lens, scale or d ** -0.5, what)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("H, HKV", [(4, 4), (8, 1), (12, 2), (32, 2), (20, 1)])
def test_decode(d, page, H, HKV):
    """One token per sequence: empty slots, one key, lengths around blocks, pages and tiles; 1 to 20
    rows for a key/value head."""
    kv = [0, 1, 2, 15, 16, 17, 127, 128, 129, 300, 0, 777]
    x = paged([1] * len(kv), kv, H, HKV, d, page, seed=page + d)
    x["q"] = x["q"].reshape(len(kv), 1, H, d)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(x, cu_seqlens=None, flags=flags)
    check_paged(got, x, [1] * len(kv), d)
    assert gdn.gdn_read_device_flags(flags) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page, H, HKV", [(16, 8, 2), (64, 6, 2), (48, 4, 4), (128, 16, 1), (32, 48, 1)])
def test_chunks_and_tokens_together(room, d, page, H, HKV):
    """Chunks of odd sizes over odd caches next to single tokens, an empty sequence and sequences
    with fewer keys than new tokens."""
    q_lens = [1, 70, 0, 1, 33, 5, 130, 9, 1, 300]
    kv = [400, 333, 50, 0, 20, 5, 130, 0, 1000, 431]
    x = paged(q_lens, kv, H, HKV, d, page, seed=page + H)
    check_paged(run(x), x, q_lens, d)


@pytest.mark.parametrize("B, T, H, HKV, d", [(3, 2, 8, 2, 64), (2, 4, 4, 1, 128), (2, 33, 16, 2, 128), (1, 515, 3, 3, 64),
                                             (3, 6, 8, 2, 128), (2, 32, 2, 2, 64), (2, 17, 2, 1, 128), (2, 1, 64, 2, 64)])
def test_equal_chunks(room, B, T, H, HKV, d):
    kv = [T + 37 * i + 5 for i in range(B)]
    x = paged([T] * B, kv, H, HKV, d, 32, seed=B + T)
    x["q"] = x["q"].reshape(B, T, H, d)
    got = run(x, cu_seqlens=None, scale=0.11)
    check_paged(got, x, [T] * B, d, scale=0.11)
    # without the log-sum-exp, into a given output, from a workspace of the queried size full of NaN
    n = gdn.gdn_attn_paged_fp8_fwd_workspace_bytes(B, T, H, HKV, d, B, 32, x["table"].shape[1])
    ws = torch.full((max(n, 4) // 4,), float("nan"), device="cuda")
    o = torch.empty_like(got[0])
    o2, lse2 = run(x, cu_seqlens=None, scale=0.11, o=o, output_lse=False, workspace=ws)
    assert lse2 is None and o2 is o and torch.equal(o2, got[0])


@pytest.mark.parametrize("nq", [1, 3, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_long_cache_is_split_and_joined(room, nq, d):
    x = paged([nq, 1], [9001, 3], 4, 1, d, 64, seed=nq)
    a, b = run(x), run(x)
    check_paged(a, x, [nq, 1], d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_token_over_very_many_keys():
    x = paged([1], [70001], 8, 1, 128, 128, seed=5)
    check_paged(run(x), x, [1], 128)


@pytest.mark.parametrize("d", [64, 128])
def test_many_units_for_each_block(room, d):
    """Far more sequences and heads than blocks, with one to nine key tiles each."""
    kv = [1 + (i * 397) % 1150 for i in range(90)]
    q_lens = [1 + (i % 3) * (i % 2) for i in range(90)]
    kv = [max(a, b) for a, b in zip(kv, q_lens)]
    x = paged(q_lens, kv, 16, 8, d, 64, seed=d)
    check_paged(run(x), x, q_lens, d)


@pytest.mark.parametrize("d, H, HKV, T", [(128, 16, 4, 1), (64, 8, 8, 1), (128, 4, 4, 3)])
@pytest.mark.parametrize("lens", ["short", "one long", "long", "whole"])
def test_many_short_sequences(d, H, HKV, T, lens):
    """Thousands of units: short ones (a warp's each), one very long sequence among them (its units
    in many pieces), longer ones (a block's each), and few enough that none is cut."""
    n = {"short": 700, "one long": 650, "long": 160, "whole": 320}[lens] * 4 // HKV
    rng = np.random.RandomState(n)
    kv = [int(x) for x in {"short": rng.randint(0, 200, n), "one long": rng.randint(1, 100, n), "long": rng.randint(700, 1400, n),
                           "whole": rng.randint(0, 500, n)}[lens]]
    if lens == "one long":
        kv[n // 2] = 9000
    x = paged([T] * n, kv, H, HKV, d, 32, seed=n + d)
    x["q"] = x["q"].reshape(n, T, H, d)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(x, cu_seqlens=None, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0
    check_paged(got, x, [T] * n, d)
    again = run(x, cu_seqlens=None)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("d, H, HKV, T, n, page", [
    (128, 32, 8, 1, 60, 64), (64, 8, 8, 8, 70, 48), (128, 16, 16, 2, 40, 16), (64, 64, 8, 1, 50, 128), (128, 24, 8, 2, 260, 64)])
def test_eight_heads_at_a_time(d, H, HKV, T, n, page):
    """Enough units of eight heads: a warp has one of them.  Empty sequences, one much longer than the others,
    malformed ones and bad pages among them; the same bits again, also on another stream and replayed."""
    rng = np.random.RandomState(n)
    kv = [int(x) for x in rng.randint(0, 1500 if n < 100 else 500, n)]
    kv[3], kv[n // 2], kv[n - 1] = 0, 6000, 1
    x = paged([T] * n, kv, H, HKV, d, page, seed=n + d)
    x["q"] = x["q"].reshape(n, T, H, d)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = run(x, cu_seqlens=None, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0
    check_paged(want, x, [T] * n, d)
    q, cache = x["q"].cuda(), device(x)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.gdn_attn_paged_fp8_fwd(q, *cache)
        with torch.cuda.graph(graph, stream=side):
            o, lse = gdn.gdn_attn_paged_fp8_fwd(q, *cache)
        for _ in range(2):
            o.fill_(7), lse.fill_(7)
            graph.replay()
            side.synchronize()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # one sequence of malformed length, and a page that is none (which reads as zeros)
    a, b = 5, n // 2 + 1
    x["lens"][a] = -3
    x["table"][b, 0] = 1 << 24
    for values in x["values"]:
        values[b][:page] = 0
    o = torch.full_like(want[0], 5.0)
    got = run(x, cu_seqlens=None, flags=flags, o=o)
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
    assert (o[a] == 5.0).all()
    rest = [i for i in range(n) if i != a]
    check([y[rest] for y in got], x["q"][rest], *([values[i] for i in rest] for values in x["values"]), [T] * len(rest), d ** -0.5)


@pytest.mark.parametrize("q_lens", [[1], [64]], ids=str)
@pytest.mark.parametrize("spread", [0.0, 12.0, 40.0])
def test_scales_far_apart(room, q_lens, spread):
    """Blocks of V that differ by up to 2^80 in size: neither the weights' sum nor what a small weight
    of a large block gives may be lost."""
    x = paged(q_lens, [611], 8, 2, 128, 32, seed=3, spread=(1.0, spread))
    check_paged(run(x), x, q_lens, 128)


@pytest.mark.parametrize("q_lens", [[1], [64]], ids=str)
def test_scales_that_are_no_powers_of_two(room, q_lens):
    """Any positive scale: a chunk's operands are rounded to bf16 then, 2^-8 of each k and v more."""
    rng = np.random.RandomState(1)

    def change(which, c, s, n):
        return c, (s * rng.uniform(0.6, 1.9, s.shape)).astype(np.float32)

    x = paged(q_lens, [333], 8, 2, 64, 16, seed=3, q_std=0.25, change=change)
    o, lse = run(x)
    ref, ref_lse, A, S = attn.attention(f64(x["q"])[0], *x["values"], q_lens, 64 ** -0.5)
    # scores are off by 2^-8 S, weights by a factor e^(2 2^-8 S) at most
    S = S.reshape(ref_lse.shape)
    assert (np.abs(f64(lse)[0] - ref_lse) <= 1.01 * 2.0 ** -8 * S + 1e-5).all()
    bound = 1.02 * ((2.0 ** -7 * S[..., None] + 2 * 2.0 ** -8) * A + 2.0 ** -8 * np.abs(ref))
    assert (np.abs(f64(o)[0] - ref) <= bound).all()


@pytest.mark.parametrize("q_lens", [[1], [50]], ids=str)
def test_blocks_of_zeros(room, q_lens):
    """Whole blocks and a whole sequence of zero values, at the smallest scale: their weights count."""
    def change(which, c, s, n):
        if which:
            c[16:200], s[1:13] = 0, 2.0 ** -117
            if n == 1:
                c[:], s[:] = 0, 2.0 ** -117
        return c, s

    q = [q_lens[0], q_lens[0]]
    x = paged(q, [300, 222], 8, 2, 128, 16, seed=11, spread=0.0, change=change)
    got = run(x)
    check_paged(got, x, q, 128)
    assert (got[0][0, q[0]:] == 0).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("q_lens", [[1], [50]], ids=str)
@pytest.mark.parametrize("rise", [4.0, -4.0, 60.0])
def test_running_maximum(room, q_lens, rise):
    """Scores that climb (or fall) along the keys, slowly and by hundreds."""
    L, H, d = 700, 2, 128
    x = paged(q_lens, [L], H, H, d, 64, seed=21)
    x["q"] = x["q"].abs()
    rng = np.random.RandomState(2)
    k = rng.randn(L, H, d) * 0.3 + rise * (np.arange(L) / L)[:, None, None]
    codes, scales, values = quantised(k, 0.0, rng)
    x["values"][0][0] = values
    for i in range(-(-L // 64)):
        pg, rows = x["table"][0, i], min(64, L - i * 64)
        x["codes"][0][pg, :rows] = codes[i * 64:i * 64 + rows]
        x["scales"][0][pg, :-(-rows // 16)] = scales[i * 4:i * 4 + -(-rows // 16)]
    check_paged(run(x), x, q_lens, d)


@pytest.mark.parametrize("std", [1e-30, 1e-6, 1e4, 1e30])
@pytest.mark.parametrize("q_lens", [[1], [40]], ids=str)
def test_size_of_queries(room, q_lens, std):
    """Queries of any size, with a scale that brings the scores back."""
    x = paged(q_lens, [200], 4, 2, 64, 16, seed=4, q_std=std)
    check_paged(run(x, scale=0.3 / std), x, q_lens, 64, scale=float(np.float32(0.3 / std)))


def test_rows_of_zeros_and_small_elements():
    """A query row of zeros weighs all keys alike; elements 2^-20 and 2^-60 of the largest one."""
    x = paged([3], [100], 4, 2, 128, 16, seed=6)
    q = x["q"]
    q[0, 0] = 0
    q[0, 1, :, 64:] *= 2.0 ** -20
    q[0, 2, :, 64:] *= 2.0 ** -60
    check_paged(run(x), x, [3], 128)


@pytest.mark.parametrize("H, HKV, q_lens, kv_lens", [
    (2, 2, [33, 40, 1], [90, 300, 7]),   # the next sequence's rows lie beside the first one's last row
    (3, 1, [35, 7, 50], [200, 20, 60]),
    (2, 2, [40, 45], [20, 30]),          # and tokens that see no key before those that see one
], ids=str)
def test_other_rows_queries_do_not_matter(room, H, HKV, q_lens, kv_lens):
    """Queries of another sequence, or of tokens that see no key, of any size: the same bits."""
    x = paged(q_lens, kv_lens, H, HKV, 64, 16, seed=8)
    want = run(x)
    check_paged(want, x, q_lens, 64)
    at = np.concatenate([[0], np.cumsum(q_lens)])
    alone = torch.zeros(at[-1], dtype=torch.bool)  # tokens whose outputs are looked at
    for n in range(0, len(q_lens), 2):
        alone[at[n] + max(q_lens[n] - kv_lens[n], 0):at[n + 1]] = True
    for size in (1e30, 1e-30, float("inf"), float("nan")):
        y = {**x, "q": x["q"].clone()}
        y["q"][0, ~alone] = (y["q"][0, ~alone].float() * size).to(torch.bfloat16)
        got = run(y)
        for a, b, what in zip(got, want, ("o", "lse")):
            assert torch.equal(a.cpu()[0, alone], b.cpu()[0, alone]), (size, what)


@pytest.mark.parametrize("nq", [1, 30])
def test_malformed_lengths_and_pages_are_flagged(room, nq):
    H, HKV, d, page = 4, 2, 64, 16
    q_lens, kv = [nq] * 3, [40, 40, 40]
    x = paged(q_lens, kv, H, HKV, d, page, seed=9)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    whole = run(x, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0
    lens = x["lens"].clone()
    for bad_len in (-1, 16 * x["table"].shape[1] + 1):  # the second sequence is left out
        x["lens"][1] = bad_len
        o = torch.full_like(whole[0], 5.0)
        run(x, flags=flags, o=o)
        assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
        assert torch.equal(o[:, :nq], whole[0][:, :nq]) and torch.equal(o[:, 2 * nq:], whole[0][:, 2 * nq:])
        assert (o[:, nq:2 * nq] == 5.0).all()
    x["lens"] = lens
    x["table"][1, 1] = 1 << 20  # a page that is none reads as zeros
    got = run(x, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
    for values in x["values"]:
        values[1][16:32] = 0
    check_paged(got, x, q_lens, d)
    # cu_seqlens that fall back
    x["cu"] = torch.tensor([0, 2 * nq, nq, 3 * nq], dtype=torch.int32)
    o = torch.full_like(whole[0], 5.0)
    run(x, flags=flags, o=o)
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS and (o == 5.0).all()


@pytest.mark.parametrize("nq", [1, 30])
def test_non_finite_values_are_reported(room, nq):
    x = paged([nq, nq], [60, 70], 4, 2, 64, 16, seed=10)
    x["codes"][1][x["table"][0, 0], 3, 1, 7] = 0x7f  # of the first sequence, second head
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, _ = run(x, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_NONFINITE
    nan = torch.isnan(o[0]).nonzero()
    assert set(map(tuple, nan.tolist())) == {(t, h, 7) for t in range(nq) for h in (2, 3)}


@pytest.mark.parametrize("nq", [1, 33])
def test_strided_queries_streams_and_graphs(room, nq):
    B, H, HKV, d = 3, 8, 2, 64
    kv = [5000, 77, 900]
    x = paged([nq] * B, kv, H, HKV, d, 16, seed=8)
    wide = normal((B, nq, H + 3, d), torch.bfloat16, 3).cuda()
    q, cache = wide[:, :, 1:H + 1], device(x)
    want = gdn.gdn_attn_paged_fp8_fwd(q.contiguous(), *cache)
    got = gdn.gdn_attn_paged_fp8_fwd(q, *cache)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x["q"] = q.cpu()
    check(want, x["q"], *x["values"], [nq] * B, d ** -0.5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    many = [gdn.gdn_attn_paged_fp8_fwd(q, *cache, stream=streams[i % 2]) for i in range(6)]  # side by side
    torch.cuda.synchronize()
    for a in many:
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.gdn_attn_paged_fp8_fwd(q, *cache)
    wide.neg_()
    graph.replay()
    again = gdn.gdn_attn_paged_fp8_fwd(q, *cache)
    torch.cuda.synchronize()
    assert torch.equal(out[0], again[0]) and not torch.equal(out[0], want[0])


def test_offsets_beyond_32_bits():
    """A cache of 5 GB, read and written near its end."""
    n_pages, page, HKV, d, H = 1 << 16, 64, 8, 128, 16
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("not enough memory")
    kc = torch.zeros((n_pages + 20000, page, HKV, d), dtype=torch.uint8, device="cuda").view(E4M3)
    vc = torch.zeros_like(kc.view(torch.uint8)).view(E4M3)
    ks = torch.zeros((n_pages + 20000, page // 16, HKV), device="cuda")
    vs = torch.zeros_like(ks)
    table = torch.tensor([[n_pages + 19999, n_pages + 7, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([170], dtype=torch.int32, device="cuda")
    k, v = (normal((1, 170, HKV, d), torch.bfloat16, s).cuda() for s in (1, 2))
    gdn.gdn_kv_cache_append_fp8(k, v, kc, vc, ks, vs, table, lens)
    rows = table[0].long()
    small = [t.view(torch.uint8)[rows].cpu().numpy() for t in (kc, vc)]
    scales = [t[rows].cpu().numpy() for t in (ks, vs)]
    empty = np.zeros((3, page, HKV, d), dtype=np.uint8)
    values = []
    for x, c, s in zip((k, v), small, scales):
        want = cache8.append(f64(x)[0], empty, np.zeros((3, page // 16, HKV), np.float32), [[0, 1, 2]], [170], [170])
        assert np.array_equal(c, want[0]) and np.array_equal(s, want[1])
        values.append(cache8.dequantise(c, s).reshape(-1, HKV, d)[:170])
    for nq in (1, 20):
        q = normal((1, nq, H, d), torch.bfloat16, 5, 2.0)
        check(gdn.gdn_attn_paged_fp8_fwd(q.cuda(), kc, vc, ks, vs, table, lens), q, [values[0]], [values[1]], [nq], d ** -0.5)
    src, dst = (torch.tensor([p], dtype=torch.int32, device="cuda") for p in (n_pages + 19999, n_pages + 11111))
    gdn.gdn_kv_cache_copy_pages(kc, vc, src, dst, k_scale=ks, v_scale=vs)
    for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs):
        assert torch.equal(t[n_pages + 11111], t[n_pages + 19999])


# ---- the write -------------------------------------------------------------------------------------------------------
def append_both(k, v, x, kv, q_lens, cu=True, flags=None):
    """The write on the GPU and by the oracle; returns the GPU's caches after they are compared."""
    dev = [t for t in device(dict(x, lens=torch.tensor(kv, dtype=torch.int32)))]
    gdn.gdn_kv_cache_append_fp8(k, v, *dev, flags=flags,
                                cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32).cuda() if cu else None)
    for i, t in enumerate((k, v)):
        want = cache8.append(f64(t).reshape(-1, *t.shape[2:]), x["codes"][i], x["scales"][i], x["table"].numpy(), kv, q_lens)
        assert np.array_equal(codes_of(dev[i]), want[0]), "codes"
        assert np.array_equal(dev[2 + i].cpu().numpy(), want[1], equal_nan=True), "scales"
    return dev


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("HKV, d, page", [(1, 64, 16), (3, 128, 48), (8, 128, 64)])
@pytest.mark.parametrize("std", [0.1, 1.0, 30.0])
def test_append(dtype, HKV, d, page, std):
    """Idle slots, fewer keys than tokens, blocks held in part whose scale has to grow (and not),
    ends inside a block; the rest of the pool keeps its bytes."""
    q_lens, kv = [1, 0, 40, 5, 1, 3, 17, 16, 1], [100, 7, 90, 5, 0, 2, 17, 32, 129]
    x = paged(q_lens, kv, HKV, HKV, d, page, seed=3)
    new = normal((1, sum(q_lens), 2 * HKV + 1, d), dtype, 77, std).cuda()
    flags = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    append_both(new[:, :, :HKV], new[:, :, HKV + 1:], x, kv, q_lens, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0


def test_append_equal_chunks_and_one_token():
    for T, kv in ((1, [16, 17, 31, 1]), (18, [18, 40, 33, 100]), (64, [64, 65, 79, 64])):
        x = paged([T] * 4, kv, 2, 2, 64, 32, seed=T)
        k, v = (normal((4, T, 2, 64), torch.bfloat16, T + i).cuda() for i in (1, 2))
        append_both(k, v, x, kv, [T] * 4, cu=False)


def test_append_token_by_token_grows_scales():
    """One token at a time with values that grow: every step equals the oracle's on what the last
    one left."""
    rng = np.random.RandomState(0)
    x = paged([1], [40], 2, 2, 64, 16, seed=1, spread=0.0)
    for n in range(1, 41):
        k, v = (normal((1, 1, 2, 64), torch.bfloat16, 2 * n + i, 0.01 * 1.3 ** n * rng.uniform(0.2, 1)).cuda() for i in (0, 1))
        dev = append_both(k, v, x, [n], [1], cu=False)
        x["codes"] = [codes_of(t).copy() for t in dev[:2]]
        x["scales"] = [t.cpu().numpy().copy() for t in dev[2:4]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_append_extreme_values(dtype):
    """Zeros, the smallest and largest numbers, ties, a block held at a scale that is no power of two."""
    kv, q_lens, HKV, d = [60], [41], 1, 64
    k, v = normal((1, 41, 1, 64), torch.float32, 1), normal((1, 41, 1, 64), torch.float32, 2)
    k[0, :13] = 0                                                  # rows 19..31: beside held rows, then a block's end
    k[0, 13:29] = torch.arange(16 * 64).view(16, 1, 64) * 0.25      # many ties
    k[0, 29:] *= 1e-40
    v[0, :13] *= 3e38 / 5
    v[0, 13:29] = 0
    v[0, 29:] *= 2.0 ** -100
    x = paged(q_lens, kv, HKV, HKV, d, 16, seed=2)
    x["scales"] = [s * np.float32(1.37) for s in x["scales"]]
    append_both(k.to(dtype).cuda(), v.to(dtype).cuda(), x, kv, q_lens)


def test_append_non_finite_values():
    x = paged([20], [30], 2, 2, 64, 16, seed=2)
    k, v = normal((1, 20, 2, 64), torch.bfloat16, 1).cuda(), normal((1, 20, 2, 64), torch.bfloat16, 2).cuda()
    k[0, 3, 0, 5], k[0, 4, 1, 6], v[0, 19, 1, 63] = float("inf"), float("-inf"), float("nan")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc = append_both(k, v, x, [30], [20], flags=flags)[0]
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_NONFINITE
    assert codes_of(kc)[x["table"][0, 0], 13, 0, 5] == 0x7f


def test_append_malformed():
    """Bad pages and lengths leave their tokens out; everything else is written."""
    q_lens, kv = [2, 20, 2], [40, 40, 40]
    x = paged(q_lens, kv, 2, 2, 64, 16, seed=9)
    k, v = (normal((1, 24, 2, 64), torch.bfloat16, i).cuda() for i in (1, 2))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def write(table, lens, cu):
        dev = list(device(x))
        dev[4], dev[5] = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        gdn.gdn_kv_cache_append_fp8(k, v, *dev, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), flags=flags)
        return [codes_of(t) for t in dev[:2]] + [t.cpu().numpy() for t in dev[2:4]]

    def equal(a, b, pages):
        return all(np.array_equal(p[pages], q[pages], equal_nan=p.dtype.kind == "f") for p, q in zip(a, b))

    before = x["codes"] + x["scales"]
    good = write(x["table"], kv, [0, 2, 22, 24])
    assert gdn.gdn_read_device_flags(flags) == 0
    own = [x["table"][n, :3].numpy() for n in range(3)]
    table = x["table"].clone()
    table[1, 1] = -5
    got = write(table, kv, [0, 2, 22, 24])
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
    assert equal(got, good, own[0]) and equal(got, good, own[2]) and equal(got, good, own[1][2:]) and equal(got, before, own[1][:2])
    for bad in (-1, 16 * x["table"].shape[1] + 1):
        got = write(x["table"], [40, bad, 40], [0, 2, 22, 24])
        assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
        assert equal(got, good, own[0]) and equal(got, good, own[2]) and equal(got, before, own[1])
    got = write(x["table"], kv, [0, 2, 30, 24])  # past the last token: nobody's
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS and equal(got, good, own[0])


def test_append_many_sequences():
    """More sequences than a warp has lanes, empty ones among them, packed."""
    rng = np.random.RandomState(4)
    q_lens = [int(n) for n in rng.choice([0, 1, 1, 2, 17, 40], 1500)]
    kv = [n + int(rng.randint(0, 40)) for n in q_lens]
    x = paged(q_lens, kv, 1, 1, 64, 16, seed=4, spread=0.0)
    k, v = (normal((1, sum(q_lens), 1, 64), torch.bfloat16, i).cuda() for i in (1, 2))
    append_both(k, v, x, kv, q_lens)


# ---- copies ----------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, E4M3], ids=str)
@pytest.mark.parametrize("page, HKV, d, n", [(16, 1, 64, 1), (48, 3, 128, 40), (64, 8, 128, 300), (16, 2, 64, 5000)])
def test_copy_pages(dtype, page, HKV, d, n):
    pool = 2 * n + 5
    gen = torch.Generator().manual_seed(n)
    bytes_ = [torch.randint(0, 256, (pool, page, HKV, d, torch.empty((), dtype=dtype).element_size()), dtype=torch.uint8,
                            generator=gen).cuda() for _ in range(2)]
    k, v = (b.view(dtype).view(pool, page, HKV, d) for b in bytes_)
    scales = [torch.rand((pool, page // 16, HKV), generator=gen).cuda() for _ in range(2)] if dtype == E4M3 else [None, None]
    perm = torch.randperm(pool, generator=gen).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    src[n // 2] = src[0]  # one source twice
    arrays = bytes_ + [s for s in scales if s is not None]
    want = [cache8_copy(a.cpu(), src, dst) for a in arrays]
    flags = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_cache_copy_pages(k, v, src.cuda(), dst.cuda(), k_scale=scales[0], v_scale=scales[1], flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0
    assert all(torch.equal(a.cpu(), w) for a, w in zip(arrays, want))


def cache8_copy(a, src, dst):
    out = a.clone()
    out[dst.long()] = a[src.long()]
    return out


@pytest.mark.parametrize("n", [6, 3000])
def test_copy_pages_that_conflict(n):
    """A destination twice, a destination that is a source, page numbers out of range: left as they
    are and reported; all other pairs are copied, whatever lies between them in the list."""
    pool, page, HKV, d = 2 * n + 10, 16, 1, 64
    gen = torch.Generator().manual_seed(n)
    k, v = (torch.randn((pool, page, HKV, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    perm = torch.randperm(pool, generator=gen).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for change in (lambda: dst.__setitem__(n - 1, int(dst[0])), lambda: dst.__setitem__(1, int(src[n - 2])),
                   lambda: src.__setitem__(2, -1), lambda: dst.__setitem__(3, pool)):
        src, dst = perm[:n].clone(), perm[n:2 * n].clone()
        change()
        kd, vd = k.cuda(), v.cuda()
        gdn.gdn_kv_cache_copy_pages(kd, vd, src.cuda(), dst.cuda(), flags=flags)
        assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
        count = {}
        for i, p in enumerate(src.tolist() + dst.tolist()):
            count.setdefault(p, set()).add(i % n)
        want_k, want_v = k.clone(), v.clone()
        for i, (s, t) in enumerate(zip(src.tolist(), dst.tolist())):
            if 0 <= s < pool and 0 <= t < pool and count[t] == {i}:
                want_k[t], want_v[t] = k[s], v[s]
        assert torch.equal(kd.cpu(), want_k) and torch.equal(vd.cpu(), want_v)
    # a page to itself, and nothing at all
    kd, vd = k.cuda(), v.cuda()
    gdn.gdn_kv_cache_copy_pages(kd, vd, perm[:3].cuda(), perm[:3].cuda(), flags=flags)
    gdn.gdn_kv_cache_copy_pages(kd, vd, perm[:0].cuda(), perm[:0].cuda())
    assert gdn.gdn_read_device_flags(flags) == 0 and torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


def test_copy_very_many_pages():
    """More pairs than blocks have room for at a time, some in conflict."""
    n, pool = 200000, 400000
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randint(0, 256, (pool, 16, 1, 64), dtype=torch.uint8, generator=gen).cuda() for _ in range(2))
    ks, vs = (torch.rand((pool, 1, 1), generator=gen).cuda() for _ in range(2))
    perm = torch.randperm(pool, generator=gen).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:].clone()
    at = torch.randperm(n, generator=gen)[:80]
    dst[at[:20]] = dst[at[20:40]]  # destinations twice
    dst[at[40:60]] = src[at[60:]]  # destinations that are sources
    good = torch.ones(n, dtype=torch.bool)
    good[at[:60]] = False
    want = []
    for a in (k, v, ks, vs):
        w = a.clone()
        w[dst[good].long().cuda()] = a[src[good].long().cuda()]
        want.append(w)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_cache_copy_pages(k.view(E4M3), v.view(E4M3), src.cuda(), dst.cuda(), k_scale=ks, v_scale=vs, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
    assert all(torch.equal(a, w) for a, w in zip((k, v, ks, vs), want))
