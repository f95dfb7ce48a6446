"""Attention over more sequences than the plan stages in shared memory (4096): lengths past those
are read where they lie.  Tolerances as derived in test_attn_gpu.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn
from test_attn_gpu import DTYPES, check_paged, paged, run_paged

pytestmark = pytest.mark.gpu


def case(dtype, packed, d=64, n=5000):
    rng = np.random.RandomState(d)
    q_lens = [int(x) for x in (rng.randint(0, 4, n) if packed else np.ones(n))]
    kv = [int(x) for x in rng.randint(0, 40, n)]
    kv[4500], kv[17] = 700, 0
    return q_lens, paged(q_lens, kv, 4, 2, d, 16, dtype, seed=5)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("packed", [False, True])
def test_thousands_of_sequences(dtype, packed):
    q_lens, x = case(DTYPES[dtype], packed)
    if not packed:
        x["q"] = x["q"].view(len(q_lens), 1, 4, 64)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_paged(x, flags=flags) if packed else run_paged(x, cu_seqlens=None, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == 0
    check_paged(got, x, q_lens, 64, DTYPES[dtype])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_malformed_behind_those_that_are_staged(dtype):
    q_lens, x = case(DTYPES[dtype], True)
    cu, T = x["cu"].clone(), sum(q_lens)
    o = torch.full((1, T, 4, 64), 77.0, dtype=DTYPES[dtype], device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    good, _ = run_paged(x)
    # one entry out of range: its two sequences are left out
    x["cu"] = cu.clone()
    x["cu"][4600] = T + 5
    run_paged(x, o=o, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS
    left_out = slice(int(cu[4599]), int(cu[4601]))
    assert (o[:, left_out] == 77.0).all()
    o[:, left_out] = good[:, left_out]
    assert torch.equal(o, good)
    # back to a token that an early sequence has: nothing is done
    x["cu"][4600] = 40
    o.fill_(77.0)
    run_paged(x, o=o, flags=flags)
    assert gdn.gdn_read_device_flags(flags) == gdn.GDN_FLAG_BAD_SEQLENS and (o == 77.0).all()
