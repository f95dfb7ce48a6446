"""The NONFINITE flag says what was written to o, whichever way it was summed."""
from __future__ import annotations

import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", [300, 3000, 9001, 70000])
def test_bf16_infinity_from_a_finite_sum(kv):
    """An output between the largest bf16 number and the largest 32-bit one, which is written as
    infinity: by the kernel itself and, from 3000 keys on, joined from three and more pieces.

    No value exceeds the largest bf16 number V, and an output is a mean of them, so only the
    roundings of the weights can take it there.  Scores and scale are such that the largest score's
    product, near 2^17, is off by 2^-9 when it is rounded for the exponents: its weight is 2^-0.0028 =
    0.998048, just above the middle between bf16's 0.99609 and 1, and counts as that in the row's sum
    and as 1 for its value; four small weights (2^-9 to 2^-12) lie just above such a middle, too.  The
    output is V (1 + .0036) / (.99805 + .0036) = 1.0019637 V, and from 511/510 V = 1.0019608 V on a
    number rounds to infinity; the unnormalised sum, 1.0036 V, is still below 2^128 = 1.0039 V."""
    d, page = 64, 64
    q = torch.zeros(d)
    q[:3] = torch.tensor([256.0, 1.0, 2.0 ** -7])
    keys = [(474, 3, 0), (474, -1, -6), (474, -1, -63), (474, -1, -122), (474, -2, -51)]  # scores of 121347 and less
    scale = float.fromhex("0x1.89c3c2p0")
    n = -(-kv // page)
    k, v = torch.zeros((n * page, d)), torch.zeros((n * page, d))
    at = kv // 2 // 128 * 128 + 5
    for i, x in enumerate(keys):
        k[at + i, :3] = torch.tensor(x, dtype=torch.float32)
        v[at + i] = torch.finfo(torch.bfloat16).max
    args = [x.to(torch.bfloat16).cuda() for x in (q.view(1, 1, 1, d), k.view(n, page, 1, d), v.view(n, page, 1, d))]
    args += [torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous(),
             torch.tensor([kv], dtype=torch.int32, device="cuda")]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = gdn.gdn_attn_paged_fwd(*args, scale=scale, flags=flags)
    assert torch.isfinite(lse).all() and torch.isinf(o).all()
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_NONFINITE


@pytest.mark.parametrize("dtype, reach", [(torch.bfloat16, 382), (torch.float32, 126)], ids=str)
@pytest.mark.parametrize("H, HKV, d", [(2, 2, 64), (1, 1, 128), (8, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("new, past, at", [(256, 0, 200), (1200, 0, 900), (1200, 0, 1023), (700, 77, 300), (90, 1001, 1080),
                                           (12, 500, 505)])
def test_a_later_value_reaches_no_further_than_its_tiles(dtype, reach, H, HKV, d, new, past, at):
    """A non-finite key or value at position `at` of a prompt's chunk over a cache (and of a whole
    prompt, where there is no past).  It is everybody's from there on.  Tokens before see it with
    weight 0, which makes NaN of a non-finite value: a token's rows are worked on with those of up to
    255 later positions (63 in fp32), over key tiles that end up to 127 (63) positions behind."""
    page, T = 16, past + new
    gen = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn((1, n, h, d), generator=gen).to(dtype).cuda() for n, h in ((new, H), (T, HKV), (T, HKV)))
    n = -(-T // page)
    table = torch.randperm(n, generator=gen).to(torch.int32)[None].cuda()
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")

    def run(k, v):
        kc, vc = (torch.full((n, page, HKV, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        gdn.gdn_kv_cache_append(k, v, kc, vc, table, lens)
        out = [gdn.gdn_attn_paged_fwd(q, kc, vc, table, lens)]
        if past == 0:
            out.append(gdn.gdn_attn_fwd(q, k, v))
        return out

    clean = run(k, v)
    row, G = at - past, H // HKV
    for x in (float("inf"), float("nan")):
        bad_k, bad_v = k.clone(), v.clone()
        bad_k[0, at, 0, 5], bad_v[0, at, 0, 5] = float("nan"), x
        for (o, lse), (o0, lse0) in zip(run(bad_k, v), clean):
            assert torch.isnan(o[0, row:, :G]).all()
            assert torch.equal(o[0, :row], o0[0, :row]) and torch.equal(o[0, row:, G:], o0[0, row:, G:])
            assert torch.equal(lse[0, :row], lse0[0, :row])
        for (o, lse), (o0, lse0) in zip(run(k, bad_v), clean):
            assert torch.equal(lse, lse0)
            assert not torch.isfinite(o[0, row:, :G, 5]).any()
            first = max(row - reach, 0)
            assert torch.equal(o[0, :first], o0[0, :first])
            o[0, first:, :G, 5] = o0[0, first:, :G, 5]
            assert torch.equal(o, o0)  # no other column, no other key/value head
