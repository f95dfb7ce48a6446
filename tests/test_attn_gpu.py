"""GPU parity of softmax attention (whole prompts, paged cache) and of the cache write against
the 64-bit definition in oracle/attn.py, through the C ABI.

Tolerances, derived from the arithmetic.  Let A = sum_j w_j |v_j| (elementwise) and
S = max_j scale sum_i |q_i k_ji| over a row's visible keys.
* A score is a sum of at most 128 products accumulated in fp32, so it is off by at most about
  2^-18 S; the log-sum-exp by as much, plus its own rounding:
  |d lse| <= 2^-18 S + 2^-20 |lse| + 1e-6.
* Scores off by e move the weights by a factor within 1 +- 2 e, the accumulation of the output in
  fp32 adds 2^-17 A: |d o| <= (2^-17 S + 2^-17) A for fp32.
* bf16 adds one rounding of each weight and one of the output.  bf16 has 8 significant bits, so a
  rounding moves a value by up to 2^-8 of it (1 + 2^-8 lies halfway between the neighbours 1 and
  1 + 2^-7): |d o| <= 2^-8 (A + |o|) * 1.01 + (2^-17 S + 2^-17) A, where the factor leaves room for
  products of the two.  Rounding errors are spread over +-2^-8 at most evenly, so each has a root
  mean square of at most 2^-8 / sqrt(3) of its value, the weights' ones fall on |v| of a column with
  random signs, and over a whole result the relative Frobenius error stays below
  sqrt(2) 2^-8 / sqrt(3) = 3.2e-3.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn
from oracle import attn

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, q, ks, vs, q_lens, scale, dtype, what=""):
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
    bound = (2.0 ** -17 * S[..., None] + 2.0 ** -17) * A
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * 1.01 * (A + np.abs(ref))
        rel = np.linalg.norm(o - ref) / max(np.linalg.norm(ref), 1e-300)
        assert rel <= 3.2e-3 or ref.size < 10000, (what, rel)  # a mean needs many values
    d = np.abs(o - ref)
    bad = d > bound
    assert not bad.any(), (what, float((d / np.maximum(bound, 1e-30)).max()), int(bad.sum()))


def packed_prompt(q_lens, H, HKV, d, dtype, seed, q_std=2.0):
    T = sum(q_lens)
    q = normal((1, T, H, d), dtype, seed, q_std)
    k, v = (normal((1, T, HKV, d), dtype, seed + i) for i in (1, 2))
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    parts = [slice(cu[i], cu[i + 1]) for i in range(len(q_lens))]
    return q, k, v, torch.tensor(cu, dtype=torch.int32), parts


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H, HKV", [(8, 8), (8, 2), (6, 2), (16, 1), (5, 1), (20, 1)])
def test_prompt_packed(dtype, d, H, HKV):
    dt = DTYPES[dtype]
    q_lens = [0, 1, 31, 64, 65, 127, 0, 128, 129, 257, 2, 300]
    q, k, v, cu, parts = packed_prompt(q_lens, H, HKV, d, dt, seed=d + H)
    got = gdn.gdn_attn_fwd(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu.cuda())
    torch.cuda.synchronize()
    check(got, q, [f64(k[0, p]) for p in parts], [f64(v[0, p]) for p in parts], q_lens, d ** -0.5, dt)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("B, T, H, HKV, d", [(1, 1, 2, 1, 64), (3, 1, 4, 2, 128), (2, 33, 16, 2, 128),
                                             (1, 1500, 2, 1, 128), (2, 515, 3, 3, 64)])
def test_prompt_batch(dtype, B, T, H, HKV, d):
    dt = DTYPES[dtype]
    q = normal((B, T, H, d), dt, 5, 2.0)
    k, v = normal((B, T, HKV, d), dt, 6), normal((B, T, HKV, d), dt, 7)
    scale = 0.11
    got = gdn.gdn_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=scale)
    check(got, q, f64(k), f64(v), [T] * B, scale, dt)
    # without the log-sum-exp, into a given output, from a workspace of the queried size full of NaN
    n = gdn.gdn_attn_fwd_workspace_bytes(B, T, H, HKV, d, B, gdn._dtype_code(dt))
    ws = torch.full((max(n, 4) // 4,), float("nan"), device="cuda")
    o = torch.empty_like(got[0])
    o2, lse2 = gdn.gdn_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=scale, o=o, output_lse=False,
                                workspace=ws)
    assert lse2 is None and o2 is o and torch.equal(o2, got[0])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_prompt_slices_of_one_projection(dtype):
    dt, B, T, H, HKV, d = DTYPES[dtype], 2, 150, 4, 2, 64
    x = normal((B, T, H + 2 * HKV + 1, d), dt, 11).cuda()  # one head of something else between
    q, k, v = x[:, :, :H], x[:, :, H:H + HKV], x[:, :, H + HKV + 1:]
    a = gdn.gdn_attn_fwd(q, k, v)
    b = gdn.gdn_attn_fwd(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(a, q.cpu(), f64(k), f64(v), [T] * B, d ** -0.5, dt)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rise", [4.0, -4.0, 60.0])
def test_running_maximum(dtype, rise):
    """Scores that climb (or fall) along the keys, slowly and by thousands: the running maximum
    moves in every tile, or never."""
    dt, T, H, d = DTYPES[dtype], 700, 2, 128
    q = normal((1, T, H, d), dt, 21).abs()
    k = normal((1, T, H, d), dt, 22, 0.3)
    k = (k + rise * (torch.arange(T)[None, :, None, None] / T)).to(dt)
    v = normal((1, T, H, d), dt, 23)
    got = gdn.gdn_attn_fwd(q.cuda(), k.cuda(), v.cuda())
    check(got, q, f64(k), f64(v), [T], d ** -0.5, dt)


def paged(q_lens, kv_lens, H, HKV, d, page, dtype, seed, spare=3, poison=True):
    """A cache whose unheld rows and pages are NaN, pages in random order, table entries past
    the last page out of range."""
    rng = np.random.RandomState(seed)
    N = len(kv_lens)
    held = [-(-n // page) for n in kv_lens]
    n_pages, width = sum(held) + spare, max(max(held), 1) + 1
    order = rng.permutation(n_pages)
    table = np.full((N, width), 1 << 30, dtype=np.int32)
    T = sum(q_lens)
    kc = torch.full((n_pages, page, HKV, d), float("nan") if poison else 0.0).to(dtype)
    vc = kc.clone()
    ks, vs, at = [], [], 0
    for n in range(N):
        k = normal((kv_lens[n], HKV, d), dtype, seed + 10 * n)
        v = normal((kv_lens[n], HKV, d), dtype, seed + 10 * n + 1)
        ks.append(k)
        vs.append(v)
        for i in range(held[n]):
            table[n, i] = order[at + i]
            rows = slice(i * page, min((i + 1) * page, kv_lens[n]))
            kc[order[at + i], :rows.stop - rows.start] = k[rows]
            vc[order[at + i], :rows.stop - rows.start] = v[rows]
        at += held[n]
    q = normal((1, T, H, d), dtype, seed + 7, 2.0)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)
    return dict(q=q, kc=kc, vc=vc, table=torch.tensor(table), cu=cu, ks=ks, vs=vs,
                lens=torch.tensor(kv_lens, dtype=torch.int32))


def run_paged(x, **kw):
    if "cu_seqlens" not in kw:
        kw["cu_seqlens"] = x["cu"].cuda()
    return gdn.gdn_attn_paged_fwd(x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), x["table"].cuda(),
                                  x["lens"].cuda(), **kw)


def check_paged(got, x, q_lens, d, dt, what=""):
    check(got, x["q"], [f64(k) for k in x["ks"]], [f64(v) for v in x["vs"]], q_lens, d ** -0.5, dt, what)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("H, HKV", [(4, 4), (8, 1), (12, 2)])
def test_decode(dtype, d, page, H, HKV):
    """One token per sequence: empty slots, one key, lengths around pages and tiles."""
    dt = DTYPES[dtype]
    kv = [0, 1, 2, 15, 16, 17, 127, 128, 129, 300, 0, 777]
    x = paged([1] * len(kv), kv, H, HKV, d, page, dt, seed=page + d)
    x["q"] = x["q"].reshape(len(kv), 1, H, d)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_paged(x, cu_seqlens=None, flags=flags)
    check_paged(got, x, [1] * len(kv), d, dt)
    assert gdn.gdn_read_device_flags(flags) == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page, H, HKV", [(16, 8, 2), (64, 6, 2), (48, 4, 4), (128, 16, 1)])
def test_chunks_and_tokens_together(dtype, d, page, H, HKV):
    """Chunks of odd sizes over odd caches next to single tokens, an empty sequence and
    sequences with fewer keys than new tokens."""
    dt = DTYPES[dtype]
    q_lens = [1, 70, 0, 1, 33, 5, 130, 9, 1, 300]
    kv = [400, 333, 50, 0, 20, 5, 130, 0, 1000, 431]
    x = paged(q_lens, kv, H, HKV, d, page, dt, seed=page + H)
    check_paged(run_paged(x), x, q_lens, d, dt)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("nq", [1, 3, 40])
def test_long_cache_is_split_and_joined(dtype, nq):
    dt, H, HKV, d = DTYPES[dtype], 4, 1, 128
    x = paged([nq, 1], [9001, 3], H, HKV, d, 64, dt, seed=nq)
    a, b = run_paged(x), run_paged(x)
    check_paged(a, x, [nq, 1], d, dt)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
def test_many_units_for_each_block(d):
    """Far more sequences and heads than blocks, with one to nine key tiles each (odd numbers next
    to even ones): every block goes through many units in a row."""
    dt, H, HKV, page = torch.bfloat16, 16, 8, 64
    kv = [1 + (i * 397) % 1150 for i in range(90)]
    q_lens = [1 + (i % 3) * (i % 2) for i in range(90)]
    kv = [max(a, b) for a, b in zip(kv, q_lens)]
    x = paged(q_lens, kv, H, HKV, d, page, dt, seed=d)
    check_paged(run_paged(x), x, q_lens, d, dt)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_append_then_attend_equals_prompt(dtype):
    """A prompt written to pages in two chunks and attended to chunk by chunk gives the whole
    prompt's attention."""
    dt, H, HKV, d, page, T, first = DTYPES[dtype], 4, 2, 64, 16, 210, 77
    q, k, v = (normal((1, T, h, d), dt, 30 + h, s).cuda() for h, s in ((H, 2.0), (HKV, 1.0), (HKV, 1.0)))
    kc = torch.full((20, page, HKV, d), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1))[:14].to(torch.int32)[None].cuda()
    outs = []
    for lo, hi in ((0, first), (first, T)):
        lens = torch.tensor([hi], dtype=torch.int32, device="cuda")
        gdn.gdn_kv_cache_append(k[:, lo:hi], v[:, lo:hi], kc, vc, table, lens)
        outs.append(gdn.gdn_attn_paged_fwd(q[:, lo:hi], kc, vc, table, lens))
    got = tuple(torch.cat([a[i] for a in outs], 1) for i in (0, 1))
    check(got, q.cpu(), f64(k), f64(v), [T], d ** -0.5, dt)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("HKV, d, page", [(1, 64, 16), (3, 128, 48), (8, 128, 64)])
def test_append(dtype, HKV, d, page):
    dt = DTYPES[dtype]
    q_lens, kv = [1, 0, 40, 5, 1, 3], [100, 7, 90, 5, 0, 2]  # an idle slot; fewer keys than tokens
    x = paged(q_lens, kv, HKV, HKV, d, page, dt, seed=3, poison=False)
    T = sum(q_lens)
    new = normal((1, T, 2 * HKV, d), dt, 77).cuda()
    k, v = new[:, :, :HKV], new[:, :, HKV:]
    kc, vc = x["kc"].cuda(), x["vc"].cuda()
    flags = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_cache_append(k, v, kc, vc, x["table"].cuda(), x["lens"].cuda(),
                            cu_seqlens=x["cu"].cuda(), flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0
    want = attn.append(f64(k)[0], f64(v)[0], f64(x["kc"]), f64(x["vc"]), x["table"].numpy(), kv, q_lens)
    assert np.array_equal(f64(kc), want[0]) and np.array_equal(f64(vc), want[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_malformed_lengths_and_pages_are_flagged(dtype):
    dt, H, HKV, d, page = DTYPES[dtype], 4, 2, 64, 16
    q_lens, kv = [2, 2, 2], [40, 40, 40]
    x = paged(q_lens, kv, H, HKV, d, page, dt, seed=9)
    good = run_paged(x)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for what in ("len", "negative", "page", "cu"):
        y = dict(x, lens=x["lens"].clone(), table=x["table"].clone(), cu=x["cu"].clone())
        if what == "len":
            y["lens"][1] = 1000
        elif what == "negative":
            y["lens"][1] = -1
        elif what == "page":
            y["table"][1, 1] = -5
        else:
            y["cu"][1] = 100
        got = run_paged(y, flags=flags)
        assert gdn.gdn_read_device_flags(flags) & gdn.GDN_FLAG_BAD_SEQLENS, what
        assert torch.equal(got[0][:, 4:], good[0][:, 4:]), what  # the last sequence is untouched
        if what == "page":
            assert torch.isfinite(got[0]).all()
        kc, vc = y["kc"].cuda(), y["vc"].cuda()
        new = normal((1, 6, HKV, d), dt, 4).cuda()
        gdn.gdn_kv_cache_append(new, new, kc, vc, y["table"].cuda(), y["lens"].cuda(),
                                cu_seqlens=y["cu"].cuda(), flags=flags)
        if what != "page":  # the appended rows are in the last page, the bad entry is not
            assert gdn.gdn_read_device_flags(flags) & gdn.GDN_FLAG_BAD_SEQLENS, what
    run_paged(x, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0  # cleared by each call


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_nonfinite_values(dtype):
    """A NaN query makes its own rows NaN and sets the flag; a NaN key or value of one sequence
    stays in that sequence; a NaN key is no concern of earlier tokens."""
    dt, d = DTYPES[dtype], 64
    q_lens = [60, 60, 300]
    q, k, v, cu, parts = packed_prompt(q_lens, 4, 2, d, dt, seed=40)
    clean = gdn.gdn_attn_fwd(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu.cuda())
    q[0, 20, 1] = float("nan")
    k[0, 80, 0, 3] = float("nan")
    v[0, 81, 1, 3] = float("inf")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = gdn.gdn_attn_fwd(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu.cuda(), flags=flags)
    assert gdn.gdn_read_device_flags(flags) & gdn.GDN_FLAG_NONFINITE
    same = torch.ones_like(o, dtype=torch.bool)
    same[0, 20, 1] = False
    same[0, 80:120, :2] = False      # query heads 0, 1 read key/value head 0
    same[0, 60:120, 2:, 3] = False   # column 3 of heads 2, 3 (earlier tokens too: the same tile)
    assert torch.isnan(o[0, 20, 1]).all() and torch.isnan(o[0, 80:120, :2]).all()
    assert not torch.isfinite(o[0, 81:120, 2:, 3]).any()
    assert torch.equal(o[same], clean[0][same])


def test_other_stream_and_graph():
    """Calls on a side stream, and a captured decode step replayed with new lengths."""
    dt, H, HKV, d, page = torch.bfloat16, 8, 2, 128, 16
    kv = [33, 500]
    x = paged([1, 1], kv, H, HKV, d, page, dt, seed=50)
    want = run_paged(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run_paged(x, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    dev = {n: t.cuda() for n, t in x.items() if torch.is_tensor(t)}
    dev["lens"] -= 1
    o = torch.empty_like(dev["q"])
    ws = torch.empty(gdn.gdn_attn_paged_fwd_workspace_bytes(1, 2, H, HKV, d, 2, page, dev["table"].shape[1],
                                                            gdn.GDN_BF16), dtype=torch.uint8, device="cuda")

    def step():
        dev["lens"] += 1
        gdn.gdn_attn_paged_fwd(dev["q"], dev["kc"], dev["vc"], dev["table"], dev["lens"],
                               cu_seqlens=dev["cu"], o=o, output_lse=False, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0])


def test_offsets_past_32_bits():
    """Pages beyond 2^31 elements of a cache (and beyond 2^32 bytes)."""
    dt, H, HKV, d, page = torch.bfloat16, 8, 8, 128, 64
    n_pages = (1 << 31) // (page * HKV * d) + 40
    kc = torch.empty((n_pages, page, HKV, d), dtype=dt, device="cuda")
    vc = torch.empty_like(kc)
    kv = 300
    table = torch.arange(n_pages - 5, n_pages, dtype=torch.int32, device="cuda")[None].contiguous()
    k, v = normal((1, kv, HKV, d), dt, 1).cuda(), normal((1, kv, HKV, d), dt, 2).cuda()
    lens = torch.tensor([kv], dtype=torch.int32, device="cuda")
    gdn.gdn_kv_cache_append(k, v, kc, vc, table, lens)
    q = normal((1, 7, H, d), dt, 3, 2.0).cuda()
    check(gdn.gdn_attn_paged_fwd(q, kc, vc, table, lens), q.cpu(), f64(k), f64(v), [7], d ** -0.5, dt)


def test_no_tokens():
    for dt in DTYPES.values():
        q, k = torch.empty((1, 0, 4, 64), dtype=dt, device="cuda"), torch.empty((1, 0, 2, 64), dtype=dt, device="cuda")
        cu = torch.zeros(3, dtype=torch.int32, device="cuda")
        o, lse = gdn.gdn_attn_fwd(q, k, k, cu_seqlens=cu)
        assert o.shape == q.shape and lse.shape == (1, 0, 4)


def test_binding_refuses_what_it_cannot_pass_on():
    x = paged([1, 1], [20, 30], 4, 2, 64, 16, torch.bfloat16, seed=1)
    d = {n: t.cuda() for n, t in x.items() if torch.is_tensor(t)}

    def call(**kw):
        args = [kw.pop(n, d[n]) for n in ("q", "kc", "vc", "table", "lens")]
        return gdn.gdn_attn_paged_fwd(*args, cu_seqlens=d["cu"], **kw)

    call()
    with pytest.raises(ValueError):
        call(q=d["q"].transpose(1, 2))
    with pytest.raises(ValueError):
        call(kc=d["kc"].float())
    with pytest.raises(ValueError):
        call(table=d["table"][:1])
    with pytest.raises(TypeError):
        call(lens=d["lens"].long())
    with pytest.raises(ValueError):
        call(vc=d["vc"][:, ::2])
    with pytest.raises(ValueError):
        call(lens=d["lens"].cpu())
    with pytest.raises(gdn.GdnError):
        call(scale=-1.0)
    with pytest.raises(gdn.GdnError):
        call(scale=float("inf"))
    with pytest.raises(gdn.GdnError):  # an output over an input
        call(o=d["q"])
    with pytest.raises(TypeError):
        gdn.gdn_attn_fwd(*(torch.zeros(1, 2, 2, 64, dtype=torch.float16, device="cuda"),) * 3)


@pytest.mark.parametrize("T, H, HKV, d", [(2500, 2, 1, 128), (6000, 1, 1, 64)])
def test_fp32_long_prompt_error(T, H, HKV, d):
    """The error of a whole fp32 result.  A score is a sum of d products in order: its partial sums
    are at most about max |s| in size, and each addition rounds by 2^-24 of them, at random, so it
    is off by about 2^-24 sqrt(d / 3) max|s|, at most 2^-24 * 6.5 * 12 = 4.6e-6 for the scores here
    in the rare largest, a third of it (1.5e-6) in a typical one; scores off by e, independently,
    move a result by about e.  T additions of the output round by 2^-24 sqrt(T / 3) = 2.7e-6 at
    most, on partial sums that are on average half of it.  A factor between two maxima, if it were
    off by the rounding of a scaled score (2^-24 * 16 = 1e-6), would add as much with each of the
    ln(T / 64) = 5 new maxima.  2e-6 holds for the first two together, not with the third."""
    q = normal((1, T, H, d), torch.float32, T, 2.0)
    k, v = normal((1, T, HKV, d), torch.float32, T + 1), normal((1, T, HKV, d), torch.float32, T + 2)
    o, _ = gdn.gdn_attn_fwd(q.cuda(), k.cuda(), v.cuda())
    ref = attn.attention(f64(q)[0], [f64(k)[0]], [f64(v)[0]], [T], d ** -0.5)[0]
    err = np.linalg.norm(f64(o)[0] - ref) / np.linalg.norm(ref)
    assert err <= 2e-6, err


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("q_lens, kv", [([257], [0]), ([1500, 2], [10, 2]), ([3000], [16])])
def test_more_new_tokens_than_keys(dtype, q_lens, kv):
    """Most tokens see no key; the pages hold far fewer positions than there are tokens."""
    dt, H, HKV, d = DTYPES[dtype], 8, 8, 128
    x = paged(q_lens, kv, H, HKV, d, 16, dt, seed=sum(q_lens))
    check_paged(run_paged(x), x, q_lens, d, dt)
