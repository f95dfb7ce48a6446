"""Refusals of the entry points of a cache in 8 bits, of page copies and of rotary positions, without
a GPU: a refused call touches no device, so fake addresses do; and the binding's own checks, on CPU
tensors."""
from __future__ import annotations

import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn
from tests.test_attn_abi import ARG, SCALE, SHAPE, UNSUPPORTED, WORKSPACE, addr, call, lib  # noqa: F401

PAGED = dict(q=addr(0), k_cache=addr(1), v_cache=addr(2), k_scale=addr(3), v_scale=addr(4), table=addr(5),
             kv_lens=addr(6), o=addr(7), lse=addr(8), cu=None, n_seqs=0, B=4, T=1, H=8, HKV=2, d=128,
             q_stride=1024, page_size=64, max_pages=100, n_pages=500, scale=0.088, dtype=1,
             flags=addr(9), ws=addr(10), ws_bytes=1 << 32)
APPEND = dict(k=addr(0), v=addr(1), k_cache=addr(2), v_cache=addr(3), k_scale=addr(4), v_scale=addr(5),
              table=addr(6), kv_lens=addr(7), cu=None, n_seqs=0, B=4, T=3, HKV=2, d=128, k_stride=256,
              v_stride=256, page_size=64, max_pages=100, n_pages=500, dtype=1, flags=addr(8))
COPY = dict(k_cache=addr(0), v_cache=addr(1), k_scale=None, v_scale=None, src=addr(2), dst=addr(3), n=40,
            HKV=2, d=128, page_size=64, n_pages=500, dtype=1, flags=addr(4))
SCALES8 = dict(k_scale=addr(5), v_scale=addr(6), dtype=2)
ROPE = dict(q=addr(0), k=addr(1), q_out=addr(2), k_out=addr(3), inv_freq=addr(4), rot=64, interleaved=0,
            mscale=1.0, kv_lens=addr(5), cu=None, n_seqs=0, B=4, T=3, H=8, HKV=2, d=128, q_stride=1024,
            k_stride=256, q_out_stride=1024, k_out_stride=256, dtype=1, flags=addr(6))
CACHE = [
    (dict(k_cache=None), ARG), (dict(v_cache=None), ARG), (dict(k_scale=None), ARG), (dict(v_scale=None), ARG),
    (dict(table=None), ARG), (dict(kv_lens=None), ARG), (dict(k_cache=addr(1, 8)), ARG),
    (dict(k_scale=addr(3, 2)), ARG), (dict(v_scale=addr(4, 1)), ARG), (dict(table=addr(5, 2)), ARG),
    (dict(kv_lens=addr(6, 1)), ARG), (dict(flags=addr(9, 2)), ARG), (dict(page_size=0), ARG),
    (dict(max_pages=0), ARG), (dict(n_pages=0), ARG), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=40), UNSUPPORTED), (dict(page_size=1 << 16, max_pages=1 << 15), UNSUPPORTED),
    (dict(page_size=1 << 12, n_pages=1 << 23), UNSUPPORTED),
]


@pytest.mark.parametrize("kw, status", SHAPE + SCALE + CACHE + [
    (dict(dtype=0), UNSUPPORTED), (dict(H=9), ARG), (dict(q=None), ARG), (dict(o=None), ARG),
    (dict(o=addr(7, 8)), ARG), (dict(lse=addr(8, 2)), ARG), (dict(q_stride=1000), ARG), (dict(q_stride=1028), ARG),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE), (dict(ws=addr(10, 128)), ARG),
    (dict(o=addr(0)), ARG), (dict(o=addr(1, 4096)), ARG), (dict(o=addr(3)), ARG), (dict(ws=addr(2)), ARG),
    (dict(lse=addr(6)), ARG), (dict(lse=addr(4)), ARG),
], ids=str)
def test_paged_refusals(lib, kw, status):  # noqa: F811
    assert call(lib.gdn_attn_paged_fp8_fwd, PAGED, kw) == status


@pytest.mark.parametrize("kw, status", SHAPE + CACHE + [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(k=addr(0, 2)), ARG), (dict(k_stride=255), ARG),
    (dict(v_stride=257), ARG), (dict(k_cache=addr(0)), ARG), (dict(v_cache=addr(2)), ARG),
    (dict(v_cache=addr(2, 4096)), ARG), (dict(table=addr(3, 64)), ARG), (dict(flags=addr(2, 64)), ARG),
    (dict(v_scale=addr(4)), ARG), (dict(k_scale=addr(2, 64)), ARG), (dict(kv_lens=addr(5, 16)), ARG),
    (dict(B=1 << 30, T=1), UNSUPPORTED),
], ids=str)
def test_append_refusals(lib, kw, status):  # noqa: F811
    assert call(lib.gdn_kv_cache_append_fp8, APPEND, kw) == status


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), ARG), (dict(HKV=0), ARG), (dict(d=0), ARG), (dict(dtype=3), ARG), (dict(d=96), UNSUPPORTED),
    (dict(HKV=1 << 16), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED), (dict(page_size=0), ARG), (dict(n_pages=0), ARG),
    (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(n=(1 << 31) - 1), UNSUPPORTED),  # each is compared with all
    (dict(k_cache=None), ARG), (dict(v_cache=None), ARG), (dict(src=None), ARG), (dict(dst=None), ARG),
    (dict(k_cache=addr(0, 8)), ARG), (dict(src=addr(2, 2)), ARG), (dict(flags=addr(4, 1)), ARG),
    (dict(dtype=2), ARG),                                       # an 8-bit cache without scales
    (dict(SCALES8, dtype=1), ARG), (dict(SCALES8, v_scale=None), ARG), (dict(SCALES8, k_scale=addr(5, 2)), ARG),
    (dict(v_cache=addr(0)), ARG), (dict(v_cache=addr(0, 64)), ARG), (dict(dst=addr(1, 64)), ARG),
    (dict(flags=addr(2)), ARG), (dict(SCALES8, v_scale=addr(5, 64)), ARG), (dict(SCALES8, src=addr(5)), ARG),
], ids=str)
def test_copy_refusals(lib, kw, status):  # noqa: F811
    assert call(lib.gdn_kv_cache_copy_pages, COPY, kw) == status


@pytest.mark.parametrize("entry", ["gdn_rope_fwd", "gdn_rope_bwd"])
@pytest.mark.parametrize("kw, status", [x for x in SHAPE if "HKV" not in x[0]] + [
    (dict(rot=0), ARG), (dict(rot=63), ARG), (dict(rot=130), ARG), (dict(rot=24), UNSUPPORTED), (dict(HKV=-1), ARG),
    (dict(HKV=1 << 16), UNSUPPORTED), (dict(interleaved=2), ARG), (dict(mscale=float("nan")), ARG), (dict(q=None), ARG),
    (dict(k=None), ARG), (dict(q_out=None), ARG), (dict(k_out=None), ARG), (dict(inv_freq=None), ARG),
    (dict(q=addr(0, 8)), ARG), (dict(k_out=addr(3, 4)), ARG), (dict(inv_freq=addr(4, 2)), ARG), (dict(kv_lens=addr(5, 2)), ARG),
    (dict(flags=addr(6, 2)), ARG), (dict(q_stride=1016), ARG), (dict(k_out_stride=260), ARG), (dict(q_out_stride=1 << 32), ARG),
    (dict(q_out=addr(0), q_out_stride=2048), ARG),              # in place at another stride
    (dict(q_out=addr(0, 16)), ARG), (dict(q_out=addr(1)), ARG), (dict(k_out=addr(2, 1024)), ARG), (dict(k_out=addr(0)), ARG),
    (dict(q_out=addr(4)), ARG), (dict(k_out=addr(5)), ARG), (dict(flags=addr(2, 64)), ARG), (dict(flags=addr(0, 64)), ARG),
    # slices of one projection's output: q's rows from 0, k's from 896 elements on would meet
    (dict(q_out=addr(0), k=addr(0, 1792), k_out=addr(0, 1792), q_stride=1280, k_stride=1280, q_out_stride=1280,
          k_out_stride=1280), ARG),
    (dict(q_out=addr(0), k=addr(0, 2304), k_out=addr(0, 2304), q_stride=1280, k_stride=1280, q_out_stride=1280,
          k_out_stride=1280), ARG),                             # k's last elements in the next token's q
], ids=str)
def test_rope_refusals(lib, entry, kw, status):  # noqa: F811
    assert call(getattr(lib, entry), ROPE, kw) == status


def test_workspace_queries(lib):  # noqa: F811
    query = gdn.gdn_attn_paged_fp8_fwd_workspace_bytes
    assert query(256, 1, 32, 8, 128, 0, 64, 64) > 0
    assert query(1, 1, 16, 2, 128, 0, 16, 20) == 0      # a short cache is not cut
    assert query(1, 1, 16, 3, 128, 0, 64, 64) == 0      # refused
    assert query(1, 1, 16, 2, 96, 0, 64, 64) == 0
    assert query(1, 1, 16, 2, 128, 0, 24, 4096) == 0
    need = query(4, 1, 8, 2, 128, 0, 64, 100)
    assert call(lib.gdn_attn_paged_fp8_fwd, PAGED, dict(ws_bytes=need - 1)) == WORKSPACE
    # more new tokens than the table holds: tiles are counted to the last one's position
    for T in (1100, 3000):  # up to 8 tiles stay whole
        assert query(1, T, 8, 8, 128, 0, 16, 1) > 0 and query(1, T, 8, 8, 128, 1, 16, 1) > 0
        kw = dict(B=1, T=T, H=8, HKV=8, page_size=16, max_pages=1, ws=None, ws_bytes=0)
        assert call(lib.gdn_attn_paged_fp8_fwd, PAGED, kw) == WORKSPACE
        assert call(lib.gdn_attn_paged_fp8_fwd, PAGED, {**kw, "cu": addr(20), "n_seqs": 1}) == WORKSPACE


def cpu(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_the_bindings_checks():
    """What the binding refuses by itself (it looks at shapes, types and devices)."""
    f8, i32, f32 = torch.float8_e4m3fn, torch.int32, torch.float32
    kc, vc, ks, vs = cpu((5, 32, 2, 64), f8), cpu((5, 32, 2, 64), f8), cpu((5, 2, 2), f32), cpu((5, 2, 2), f32)
    table, lens, q, k = cpu((3, 2), i32), cpu((3,), i32), cpu((3, 1, 4, 64)), cpu((3, 1, 2, 64))
    cache = dict(k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, block_table=table, kv_lens=lens)
    wrong = [dict(k_cache=kc.view(torch.uint8)), dict(v_cache=cpu((5, 32, 2, 128), f8)), dict(k_scale=cpu((5, 32, 2), f32)),
             dict(v_scale=cpu((5, 2, 2))), dict(v_scale=cpu((5, 2, 3), f32)), dict(block_table=cpu((4, 2), i32)),
             dict(kv_lens=cpu((3,), torch.int64)), dict(k_scale=cpu((5, 2, 4), f32)[:, :, ::2])]
    for kw in wrong:
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_attn_paged_fp8_fwd(q, **{**cache, **kw})
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_kv_cache_append_fp8(k, k, **{**cache, **kw})
    pages = cpu((2,), i32)
    for kw in (dict(), dict(k_scale=ks), dict(k_scale=ks, v_scale=vs, src=cpu((3,), i32)), dict(k_scale=ks, v_scale=vs, src=cpu((2,), torch.int64)),
               dict(k_scale=ks, v_scale=vs, v_cache=cpu((5, 32, 2, 64))), dict(k_cache=cpu((5, 32, 2, 64)), v_cache=cpu((5, 32, 2, 64)), k_scale=ks, v_scale=vs)):
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_kv_cache_copy_pages(**{**dict(k_cache=kc, v_cache=vc, src=pages, dst=pages), **kw})
    freq = cpu((16,), f32)
    for kw in (dict(k=cpu((3, 1, 2, 128))), dict(k=cpu((3, 2, 2, 64))), dict(k=cpu((3, 1, 2, 64), f32)), dict(inv_freq=cpu((16,))),
               dict(inv_freq=cpu((4, 4), f32)), dict(kv_lens=cpu((2,), i32)), dict(kv_lens=cpu((3,), f32)), dict(q_out=cpu((3, 1, 5, 64))),
               dict(q_out=cpu((3, 1, 4, 64), f32)), dict(k=None, k_out=k), dict(q=cpu((3, 4, 64)))):
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_rope_fwd(**{**dict(q=q, k=k, inv_freq=freq), **kw})
