"""Tensors in host memory are refused by the binding before anything is launched, also where a stream is given (its
device says nothing about the tensors).  Without a GPU: the stream is a stand-in."""
from __future__ import annotations

import types

import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import gdn

STREAM = types.SimpleNamespace(cuda_stream=0)
BF16, F32, I32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=torch.uint8 if dtype is E4M3 else dtype).view(dtype) if dtype is E4M3 else torch.zeros(shape, dtype=dtype)


K, TABLE, LENS = zeros(1, 4, 1, 64), zeros(1, 1, dtype=I32), torch.full((1,), 4, dtype=I32)
G = zeros(1, 4, 1, dtype=F32)


def caches(dtype):
    return zeros(2, 16, 1, 64, dtype=dtype), zeros(2, 16, 1, 64, dtype=dtype)


def scales():
    return zeros(2, 1, 1, dtype=F32), zeros(2, 1, 1, dtype=F32)


CALLS = dict(
    append8=lambda: gdn.gdn_kv_cache_append_fp8(K, K.clone(), *caches(E4M3), *scales(), TABLE, LENS, stream=STREAM),
    append=lambda: gdn.gdn_kv_cache_append(K, K.clone(), *caches(BF16), TABLE, LENS, stream=STREAM),
    copy=lambda: gdn.gdn_kv_cache_copy_pages(*caches(BF16), zeros(1, dtype=I32), zeros(1, dtype=I32) + 1, stream=STREAM),
    chunk=lambda: gdn.gdn_chunk_fwd(K.repeat(1, 1, 1, 2), K.repeat(1, 1, 1, 2), K.repeat(1, 1, 1, 2), G, G, stream=STREAM),
    recurrent=lambda: gdn.gdn_recurrent_fwd(K, K, K, G, G, stream=STREAM),
    l2norm=lambda: gdn.gdn_l2norm_fwd(K, stream=STREAM),
)


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_does_not_make_them_device_tensors(name):
    with pytest.raises(ValueError, match="on a GPU"):
        CALLS[name]()
