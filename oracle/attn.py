"""Plain 64-bit softmax attention over a list of sequences and a plain paged-cache write, in
numpy, for the tests: the definition, one head at a time, with the quantities that the error
bounds of the tests are made of."""
from __future__ import annotations

import numpy as np


def attention(q, ks, vs, q_lens, scale):
    """q [Ttot, H, d]; ks, vs: per sequence [L, HKV, d], the new tokens as the last keys.

    Returns (o [Ttot, H, d], lse [Ttot, H], weighted [Ttot, H, d], spread [Ttot, H]):
    ``weighted`` is sum_j w_j |v_j| and ``spread`` the largest scale * sum_i |q_i k_ji| over
    the visible keys.  A token without a visible key has o = 0 and lse = -inf.
    """
    q = np.asarray(q, dtype=np.float64)
    Ttot, H, d = q.shape
    o, weighted = np.zeros((Ttot, H, d)), np.zeros((Ttot, H, d))
    lse, spread = np.full((Ttot, H), -np.inf), np.zeros((Ttot, H))
    at = 0
    for nq, k, v in zip(q_lens, ks, vs):
        k, v = np.asarray(k, dtype=np.float64), np.asarray(v, dtype=np.float64)
        L, HKV = k.shape[:2]
        for t in range(nq):
            end = L - nq + t + 1  # keys that token t sees
            if end <= 0:
                continue
            for h in range(HKV):
                hs = slice(h * (H // HKV), (h + 1) * (H // HKV))
                x = q[at + t, hs]
                s = scale * (x @ k[:end, h].T)
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                l = e.sum(-1, keepdims=True)
                w = e / l
                o[at + t, hs] = w @ v[:end, h]
                weighted[at + t, hs] = w @ np.abs(v[:end, h])
                lse[at + t, hs] = (m + np.log(l))[:, 0]
                spread[at + t, hs] = scale * (np.abs(x) @ np.abs(k[:end, h]).T).max(-1)
        at += nq
    return o, lse, weighted, spread


def append(k, v, k_cache, v_cache, table, kv_lens, q_lens):
    """Write rows of k, v [Ttot, HKV, d] into copies of the caches; returns them."""
    k_cache, v_cache = np.array(k_cache), np.array(v_cache)
    page = k_cache.shape[1]
    at = 0
    for n, nq in enumerate(q_lens):
        for t in range(nq):
            p = int(kv_lens[n]) - nq + t
            if p >= 0:
                k_cache[table[n][p // page], p % page] = k[at + t]
                v_cache[table[n][p // page], p % page] = v[at + t]
        at += nq
    return k_cache, v_cache
