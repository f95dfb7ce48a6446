"""Refusals of the attention and cache entry points of the C ABI, without a GPU: a refused call
touches no device, so fake addresses do."""
from __future__ import annotations

import ctypes

import pytest

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build
from chunkwise_gated_delta_gdn_gb300 import gdn

ARG, UNSUPPORTED, WORKSPACE = (gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED,
                               gdn.GDN_ERR_WORKSPACE)
BASE, STRIDE = 1 << 40, 1 << 36
INT_MAX = 2 ** 31 - 1


def addr(i, off=0):
    return ctypes.c_void_p(BASE + i * STRIDE + off)


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return gdn.load()


PROMPT = dict(q=addr(0), k=addr(1), v=addr(2), o=addr(3), lse=addr(4), cu=None, n_seqs=0, B=2,
              T=20000, H=8, HKV=2, d=128, q_stride=1024, k_stride=256, v_stride=256, scale=0.088,
              dtype=1, flags=addr(5), ws=addr(6), ws_bytes=1 << 32)
CUT = dict(H=2, T=5000)  # few and long units, cut between blocks: only then is a workspace asked for
PAGED = dict(q=addr(0), k_cache=addr(1), v_cache=addr(2), table=addr(3), kv_lens=addr(4),
             o=addr(5), lse=addr(6), cu=None, n_seqs=0, B=4, T=1, H=8, HKV=2, d=128, q_stride=1024,
             page_size=64, max_pages=100, n_pages=500, scale=0.088, dtype=1, flags=addr(7),
             ws=addr(8), ws_bytes=1 << 32)
APPEND = dict(k=addr(0), v=addr(1), k_cache=addr(2), v_cache=addr(3), table=addr(4),
              kv_lens=addr(5), cu=None, n_seqs=0, B=4, T=3, HKV=2, d=128, k_stride=256,
              v_stride=256, page_size=64, max_pages=100, n_pages=500, dtype=1, flags=addr(6))

SHAPE = [
    (dict(B=0), ARG),
    (dict(T=-1), ARG),
    (dict(HKV=0), ARG),
    (dict(d=0), ARG),
    (dict(dtype=2), ARG),
    (dict(n_seqs=3), ARG),                       # neither 0 nor B
    (dict(cu=addr(20), n_seqs=2), ARG),          # packed needs B == 1
    (dict(cu=addr(20), B=1, n_seqs=0), ARG),
    (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED),
    (dict(B=1 << 15, T=1 << 16), UNSUPPORTED),   # tokens are counted in 32 bits
]
CACHE = [
    (dict(k_cache=None), ARG),
    (dict(v_cache=None), ARG),
    (dict(table=None), ARG),
    (dict(kv_lens=None), ARG),
    (dict(k_cache=addr(1, 8)), ARG),
    (dict(table=addr(3, 2)), ARG),
    (dict(kv_lens=addr(4, 1)), ARG),
    (dict(flags=addr(7, 2)), ARG),
    (dict(page_size=0), ARG),
    (dict(max_pages=0), ARG),
    (dict(n_pages=0), ARG),
    (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=40), UNSUPPORTED),
    (dict(page_size=1 << 16, max_pages=1 << 15), UNSUPPORTED),
    (dict(page_size=1 << 12, n_pages=1 << 23), UNSUPPORTED),
]
SCALE = [(dict(scale=x), ARG) for x in (0.0, -1.0, float("inf"), float("nan"))]


def call(entry, base, kw):
    """`base` is in the order of the entry's arguments."""
    return entry(*{**base, **kw}.values(), None)


@pytest.mark.parametrize("kw, status", SHAPE + SCALE + [
    (dict(H=9), ARG),                            # not a multiple of HKV
    (dict(H=0), ARG),
    (dict(q=None), ARG),
    (dict(k=None), ARG),
    (dict(v=None), ARG),
    (dict(o=None), ARG),
    (dict(q=addr(0, 8)), ARG),
    (dict(o=addr(3, 4)), ARG),
    (dict(lse=addr(4, 2)), ARG),
    (dict(flags=addr(5, 1)), ARG),
    (dict(q_stride=1016), ARG),                  # less than a token
    (dict(k_stride=260), ARG),                   # not a multiple of 16 bytes
    (dict(v_stride=1 << 32), ARG),
    (dict(ws=None, **CUT), WORKSPACE),
    (dict(ws_bytes=1000, **CUT), WORKSPACE),
    (dict(ws=addr(6, 16)), ARG),
    (dict(o=addr(0)), ARG),                      # output over an input
    (dict(o=addr(2, 256)), ARG),
    (dict(lse=addr(3, 1024)), ARG),              # output over an output
    (dict(ws=addr(1), **CUT), ARG),
    (dict(flags=addr(6), **CUT), ARG),           # status word inside the workspace
], ids=str)
def test_prompt_refusals(lib, kw, status):
    assert call(lib.gdn_attn_fwd, PROMPT, kw) == status


@pytest.mark.parametrize("kw, status", SHAPE + SCALE + CACHE + [
    (dict(H=9), ARG),
    (dict(q=None), ARG),
    (dict(o=None), ARG),
    (dict(o=addr(5, 8)), ARG),
    (dict(lse=addr(6, 2)), ARG),
    (dict(q_stride=1000), ARG),
    (dict(q_stride=1028), ARG),
    (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=1000), WORKSPACE),
    (dict(ws=addr(8, 128)), ARG),
    (dict(o=addr(0)), ARG),
    (dict(o=addr(1, 4096)), ARG),                # an output inside the cache
    (dict(ws=addr(2)), ARG),
    (dict(lse=addr(4)), ARG),
], ids=str)
def test_paged_refusals(lib, kw, status):
    assert call(lib.gdn_attn_paged_fwd, PAGED, kw) == status


@pytest.mark.parametrize("kw, status", SHAPE + CACHE + [
    (dict(k=None), ARG),
    (dict(v=None), ARG),
    (dict(k=addr(0, 2)), ARG),
    (dict(k_stride=255), ARG),
    (dict(v_stride=257), ARG),
    (dict(k_cache=addr(0)), ARG),                # the cache over the new keys
    (dict(v_cache=addr(2)), ARG),                # one cache for both
    (dict(v_cache=addr(2, 4096)), ARG),
    (dict(table=addr(3, 64)), ARG),              # the table inside a cache
    (dict(flags=addr(2, 64)), ARG),
], ids=str)
def test_append_refusals(lib, kw, status):
    assert call(lib.gdn_kv_cache_append, APPEND, kw) == status


def test_workspace_queries(lib):
    prompt = gdn.gdn_attn_fwd_workspace_bytes
    paged = gdn.gdn_attn_paged_fwd_workspace_bytes
    # 2 partial results of 256 rows per block (64 in fp32), each row d + 2 floats, and 32 bytes
    # per block: 152 blocks of bf16, 2 or 3 per processor in fp32 (also where no GPU is present)
    for d in (64, 128):
        part = 2 * 256 * (d + 2) * 4 + 32
        for need in (prompt(1, 8192, 32, 8, d, 4, gdn.GDN_BF16), prompt(1, 20000, 1, 1, d, 0, gdn.GDN_BF16),
                     prompt(2, 5000, 2, 2, d, 0, gdn.GDN_BF16)):
            assert need % part == 0 and need > 0
        part = 2 * 64 * (d + 2) * 4 + 32
        assert prompt(4, 2048, 32, 8, d, 0, gdn.GDN_F32) % part == 0
    assert paged(256, 1, 32, 8, 128, 0, 64, 64, gdn.GDN_BF16) > 0
    # nothing can be cut, so nothing is stored: few short prompts, short caches
    assert prompt(1, 33, 16, 2, 128, 0, gdn.GDN_BF16) == 0
    assert paged(1, 1, 16, 2, 128, 0, 16, 20, gdn.GDN_BF16) == 0
    # equal prompts with enough units for each block: dealt whole
    assert prompt(4, 2048, 32, 8, 128, 0, gdn.GDN_BF16) == 0
    # what the entry points refuse needs nothing
    assert prompt(1, 4096, 16, 3, 128, 0, gdn.GDN_BF16) == 0
    assert prompt(1, 4096, 16, 2, 96, 0, gdn.GDN_BF16) == 0
    assert paged(1, 1, 16, 2, 128, 0, 24, 4096, gdn.GDN_BF16) == 0
    # a few more sequences never need less: blocks have the same parts whatever they hold
    assert prompt(1, 32768, 16, 2, 128, 0, 1) == prompt(1, 8192, 32, 8, 128, 4, 1)


def test_query_covers_what_the_call_asks_for(lib):
    """One byte less than the query's answer is refused for the same shape, unless the query had
    to cover another form of it (one sequence, with and without cu_seqlens)."""
    for kw in (CUT, dict(T=5170, d=64, **{"H": 2}), dict(dtype=0, T=3000), dict(dtype=0, B=70, T=1024)):
        a = {**PROMPT, **kw}
        a.update(q_stride=a["H"] * a["d"], k_stride=a["HKV"] * a["d"], v_stride=a["HKV"] * a["d"])
        need = gdn.gdn_attn_fwd_workspace_bytes(a["B"], a["T"], a["H"], a["HKV"], a["d"], 0,
                                                a["dtype"])
        assert need > 0
        assert call(lib.gdn_attn_fwd, a, dict(ws_bytes=need - 1)) == WORKSPACE
    need = gdn.gdn_attn_paged_fwd_workspace_bytes(4, 1, 8, 2, 128, 0, 64, 100, 1)
    assert call(lib.gdn_attn_paged_fwd, PAGED, dict(ws_bytes=need - 1)) == WORKSPACE


@pytest.mark.parametrize("dtype, T", [(0, 257), (1, 3000)])
def test_more_new_tokens_than_the_table_holds(lib, dtype, T):
    """A table of one page and many new tokens (most see no key): the plan counts tiles up to the
    last token's position and may cut them, so there has to be a workspace."""
    assert gdn.gdn_attn_paged_fwd_workspace_bytes(1, T, 8, 8, 128, 0, 16, 1, dtype) > 0
    assert gdn.gdn_attn_paged_fwd_workspace_bytes(1, T, 8, 8, 128, 1, 16, 1, dtype) > 0
    kw = dict(B=1, T=T, H=8, HKV=8, page_size=16, max_pages=1, dtype=dtype, ws=None, ws_bytes=0)
    assert call(lib.gdn_attn_paged_fwd, PAGED, kw) == WORKSPACE
    assert call(lib.gdn_attn_paged_fwd, PAGED, {**kw, "cu": addr(20), "n_seqs": 1}) == WORKSPACE
