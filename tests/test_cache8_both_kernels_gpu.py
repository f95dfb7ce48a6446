"""Calls of attention over a cache in 8 bits that have chunks and single tokens at once, and so two kernels of which the second
begins while the first one ends, and two joinings: captured and replayed on inputs that change, one behind the other on one
workspace, and side by side on two streams."""
from __future__ import annotations

import pytest
import torch

from tests.test_cache8_gpu import check_paged, device, gdn, paged

pytestmark = pytest.mark.gpu

Q_LENS = [1, 300, 1, 70, 1, 1, 0, 40]
KV = [9000, 5000, 17, 6000, 700, 1, 300, 4000]
SHAPES = [(8, 2, 128, 64), (32, 4, 64, 32)]


def make(H, HKV, d, page, seeds=(1, 2, 3)):
    return [paged(Q_LENS, KV, H, HKV, d, page, seed=s) for s in seeds]


def arguments(x):
    return [x["q"].cuda(), *device(x)], x["cu"].cuda()


@pytest.fixture
def long_table():
    """Room for 2^18 positions: the call is not a small one that one kernel does."""
    import tests.test_cache8_gpu as base
    base._room = 1 << 18
    yield
    base._room = 0


@pytest.mark.parametrize("H, HKV, d, page", SHAPES)
def test_captured_and_replayed(long_table, H, HKV, d, page):
    xs = make(H, HKV, d, page)
    calls = [arguments(x) for x in xs]
    want = []
    for (args, cu), x in zip(calls, xs):
        want.append(gdn.gdn_attn_paged_fp8_fwd(*args, cu_seqlens=cu))
        check_paged(want[-1], x, Q_LENS, d)
    held = [t.clone() for t in calls[0][0]]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = gdn.gdn_attn_paged_fp8_fwd(*held, cu_seqlens=calls[0][1], flags=flags)
    for i in (0, 1, 2, 1, 0):
        for t, new in zip(held, calls[i][0]):
            t.view(torch.uint8).copy_(new.view(torch.uint8))
        o.fill_(7), lse.fill_(7)
        for _ in range(3):  # one replay behind the other
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]), i
        assert gdn.gdn_read_device_flags(flags) == 0


@pytest.mark.parametrize("H, HKV, d, page", SHAPES)
def test_one_behind_the_other_on_one_workspace(long_table, H, HKV, d, page):
    xs = make(H, HKV, d, page)
    calls = [arguments(x) for x in xs]
    want = [gdn.gdn_attn_paged_fp8_fwd(*args, cu_seqlens=cu) for args, cu in calls]
    width = xs[0]["table"].shape[1]
    n = gdn.gdn_attn_paged_fp8_fwd_workspace_bytes(1, sum(Q_LENS), H, HKV, d, len(KV), page, width)
    assert n > 0
    ws = torch.full((n // 4,), float("nan"), device="cuda")
    got = []
    for i in range(12):
        args, cu = calls[i % 3]
        got.append(gdn.gdn_attn_paged_fp8_fwd(*args, cu_seqlens=cu, workspace=ws))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(lse, want[i % 3][1]), i


@pytest.mark.parametrize("H, HKV, d, page", SHAPES)
def test_side_by_side_on_two_streams(long_table, H, HKV, d, page):
    xs = make(H, HKV, d, page)
    calls = [arguments(x) for x in xs]
    want = [gdn.gdn_attn_paged_fp8_fwd(*args, cu_seqlens=cu) for args, cu in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(12):
        args, cu = calls[i % 3]
        got.append(gdn.gdn_attn_paged_fp8_fwd(*args, cu_seqlens=cu, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(lse, want[i % 3][1]), i


@pytest.mark.parametrize("H, HKV, d, page", SHAPES)
def test_what_follows_sees_both_kernels_outputs(long_table, H, HKV, d, page):
    """A copy queued right behind the call, on the same stream, has every output."""
    (x,) = make(H, HKV, d, page, seeds=(4,))
    args, cu = arguments(x)
    want = gdn.gdn_attn_paged_fp8_fwd(*args, cu_seqlens=cu)
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    copies = []
    for _ in range(10):
        o.fill_(7), lse.fill_(7)
        gdn.gdn_attn_paged_fp8_fwd(*args, cu_seqlens=cu, o=o, lse=lse)
        copies.append((o.clone(), lse.clone()))
    torch.cuda.synchronize()
    for a, b in copies:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
