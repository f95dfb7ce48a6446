"""cu_seqlens that fall back behind an earlier sequence's end: attention does nothing but report
them.  (tests/test_attn_plan_calls.py goes through the plan of such calls on the CPU.)"""
from __future__ import annotations

import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn

pytestmark = pytest.mark.gpu


def calls(cu, T, H, HKV, d, dtype):
    """The prompt's and the paged attention with these cu_seqlens, as (o, lse, flags) filled with
    a number that no result is."""
    gen = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn((1, T, h, d), generator=gen).to(dtype).cuda() for h in (H, HKV, HKV))
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    n, page = cu.numel() - 1, 64
    held = -(-T // page)
    kc, vc = (x.new_zeros((held, page, HKV, d)) for x in (k, v))
    table = torch.arange(held, dtype=torch.int32, device="cuda").repeat(n, 1)
    lens = torch.full((n,), T, dtype=torch.int32, device="cuda")
    for paged in (False, True):
        o, lse = torch.full_like(q, 77.0), torch.full((1, T, H), 77.0, device="cuda")
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        if paged:
            gdn.gdn_attn_paged_fwd(q, kc, vc, table, lens, cu_seqlens=cu, o=o, lse=lse, flags=flags)
        else:
            gdn.gdn_attn_fwd(q, k, v, cu_seqlens=cu, o=o, lse=lse, flags=flags)
        yield o, lse, gdn.gdn_read_device_flags(flags)


@pytest.mark.parametrize("cu, T, H, HKV, d, dtype", [
    ([0, 900] * 3, 900, 4, 1, 128, torch.bfloat16),
    ([0, 600] * 3, 600, 20, 20, 64, torch.bfloat16),
    ([0, 1000] * 4, 1000, 8, 8, 128, torch.bfloat16),
    ([0, 120] * 20, 120, 2, 1, 64, torch.float32),
    ([0, 300, 5000, 0, 300, 600], 600, 4, 2, 128, torch.bfloat16),  # back by way of an entry out of range
    ([0, 300, 290, 600], 600, 4, 2, 64, torch.float32),
], ids=str)
def test_falling_back(cu, T, H, HKV, d, dtype):
    for o, lse, flags in calls(cu, T, H, HKV, d, dtype):
        assert flags == gdn.GDN_FLAG_BAD_SEQLENS
        assert (o == 77.0).all() and (lse == 77.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_one_entry_out_of_range(dtype):
    """The two sequences beside it are left out, the others stay."""
    good = list(calls([0, 40, 90, 200, 300], 300, 4, 2, 64, dtype))
    for bad in (-1, 301, 1 << 30, -2 ** 31, 2 ** 31 - 1):
        for (o, lse, flags), (o0, lse0, none) in zip(calls([0, 40, bad, 200, 300], 300, 4, 2, 64, dtype), good):
            assert flags == gdn.GDN_FLAG_BAD_SEQLENS and none == 0
            for x, x0 in ((o, o0), (lse, lse0)):
                assert (x[:, 40:200] == 77.0).all()
                assert torch.equal(x[:, :40], x0[:, :40]) and torch.equal(x[:, 200:], x0[:, 200:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("cu, written", [
    ([0, 6, 0, 6], 6),                     # each token is in the first sequence
    ([0, 2, 2, 2, 1, 6], 6),               # back by one
    ([0, 6] + [0] * 40 + [6], 6),
    ([0, 4, 4, 3], 4),                     # the last two tokens belong to nobody
], ids=str)
def test_cache_write_reports_malformed_sequences(dtype, cu, written):
    """Also where every token finds a sequence that is well formed by itself."""
    HKV, d, page, T, n = 2, 64, 16, 6, len(cu) - 1
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn((1, T, HKV, d), generator=gen).to(dtype).cuda() for _ in range(2))
    kc, vc = torch.zeros((n, page, HKV, d), dtype=dtype, device="cuda"), torch.zeros((n, page, HKV, d), dtype=dtype, device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.full((n,), T, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_cache_append(k, v, kc, vc, table, lens, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            flags=flags)
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
    for cache, new in ((kc, k), (vc, v)):  # each token once, no others
        rows = cache.flatten(0, 1).flatten(1)
        rows = rows[rows.any(1)]
        assert len(rows) == written
        assert all((rows == x).all(1).any() for x in new[0, :written].flatten(1))
