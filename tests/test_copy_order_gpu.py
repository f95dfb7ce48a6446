"""Page copies whose destinations lie in order or evenly spaced, as where a pool is put in order: conflicts among them are found
as among shuffled ones."""
from __future__ import annotations

import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("apart, n", [(1, 20000), (2, 20000), (64, 3000), (256, 3000)])
@pytest.mark.parametrize("conflicts", [False, True])
def test_destinations_in_order(apart, n, conflicts):
    pool = n * apart + n
    gen = torch.Generator().manual_seed(apart)
    k, v = (torch.randint(0, 256, (pool, 16, 1, 64), dtype=torch.uint8, generator=gen).cuda().view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.rand((pool, 1, 1), generator=gen).cuda() for _ in range(2))
    dst = torch.arange(n, dtype=torch.int32) * apart
    src = n * apart + torch.randperm(n, generator=gen).to(torch.int32)
    good = torch.ones(n, dtype=torch.bool)
    if conflicts:
        at = torch.randperm(n, generator=gen)[:40]
        dst[at[:10]] = dst[at[10:20]]  # destinations twice
        src[at[20:30]] = dst[at[30:]]  # sources that are destinations
        good[at[:20]] = good[at[30:]] = False
    want = []
    for t in (k.view(torch.uint8), v.view(torch.uint8), ks, vs):
        w = t.clone()
        w[dst[good].long().cuda()] = t[src[good].long().cuda()]
        want.append(w)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_cache_copy_pages(k, v, src.cuda(), dst.cuda(), k_scale=ks, v_scale=vs, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == (gdn.GDN_FLAG_BAD_SEQLENS if conflicts else 0)
    for t, w in zip((k.view(torch.uint8), v.view(torch.uint8), ks, vs), want):
        assert torch.equal(t, w)
