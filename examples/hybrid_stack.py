"""A small stack of gated-delta and softmax-attention layers, served as such stacks are: a packed
prefill of prompts of different lengths, then one token per sequence and step.

    python examples/hybrid_stack.py

Layers are given as a string, "G" for a gated-delta layer (projection, causal convolution, L2 norm
of q and k, recurrence, gated RMS norm) and "A" for an attention layer with grouped heads over a
paged cache; each adds to its input.  Weights are random.  A gated-delta layer keeps a state of
fixed size per sequence, an attention layer its keys and values in pages that any sequence may hold.
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunkwise_gated_delta_gdn_gb300 import gdn  # noqa: E402

WIDTH = 256                # of the stream between layers
H, HV, DK = 2, 4, 128      # gated-delta layer: key and value heads, head size
AH, AHKV, AD = 8, 2, 64    # attention layer: query and key/value heads, head size
TAPS, PAGE = 4, 16


def rms(x):
    return F.rms_norm(x, (x.shape[-1],))


class Stack:
    def __init__(self, layers="GGAG", dtype=torch.bfloat16, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)

        def weight(rows, cols, std=None, dt=dtype):
            w = torch.randn((rows, cols), generator=gen) * (std or rows ** -0.5)
            return w.to(device=device, dtype=dt)

        self.dtype, self.device, self.layers = dtype, device, []
        for kind in layers:
            if kind == "A":
                p = dict(qkv=weight(WIDTH, (AH + 2 * AHKV) * AD), out=weight(AH * AD, WIDTH))
            else:
                conv = (2 * H + HV) * DK
                p = dict(qkv=weight(WIDTH, conv), z=weight(WIDTH, HV * DK), gate=weight(WIDTH, 2 * HV),
                         taps=weight(conv, TAPS, 0.5, torch.float32), out=weight(HV * DK, WIDTH),
                         norm=torch.ones(DK, device=device))
            self.layers.append((kind, p))

    def allocate(self, n_seqs, max_len):
        """An empty cache for each layer, and the pages that the sequences hold: here each
        sequence's are given to it at once, in no order."""
        dev, per = self.device, -(-max_len // PAGE)
        self.table = torch.randperm(n_seqs * per).to(torch.int32).view(n_seqs, per).to(dev)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
        self.cache = []
        for kind, _ in self.layers:
            if kind == "A":
                pages = torch.zeros((2, n_seqs * per, PAGE, AHKV, AD), dtype=self.dtype, device=dev)
                self.cache.append((pages[0], pages[1]))
            else:
                self.cache.append((torch.zeros((n_seqs, (2 * H + HV) * DK, TAPS - 1), device=dev),
                                   torch.zeros((n_seqs, HV, DK, DK), device=dev)))

    def delta(self, p, x, cache, cu):
        history, state = cache
        B, T = x.shape[:2]
        y, _ = gdn.gdn_causal_conv1d_fwd(x @ p["qkv"], p["taps"], None, history, cu_seqlens=cu,
                                         hT=history, activation=gdn.GDN_ACT_SILU)
        q, k, v = y.split([H * DK, H * DK, HV * DK], -1)
        q = gdn.gdn_l2norm_fwd(q.contiguous().view(B, T, H, DK))
        k = gdn.gdn_l2norm_fwd(k.contiguous().view(B, T, H, DK))
        v = v.contiguous().view(B, T, HV, DK)
        a, b = (x @ p["gate"]).float().chunk(2, -1)
        g, beta = -F.softplus(a), torch.sigmoid(b)
        if T == 1 and cu is None:
            o, _ = gdn.gdn_recurrent_fwd(q, k, v, g, beta, state, hT=state)
        else:
            o, last = gdn.gdn_chunk_fwd(q, k, v, g, beta, state, cu_seqlens=cu)
            state.copy_(last)
        z = (x @ p["z"]).view(B, T, HV, DK)
        return gdn.gdn_rmsnorm_gated_fwd(o, p["norm"], z).view(B, T, HV * DK) @ p["out"]

    def attention(self, p, x, cache, cu, whole):
        k_cache, v_cache = cache
        B, T = x.shape[:2]
        # slices of the projection: their tokens lie (AH + 2 AHKV) AD elements apart
        q, k, v = (x @ p["qkv"]).view(B, T, AH + 2 * AHKV, AD).split([AH, AHKV, AHKV], 2)
        gdn.gdn_kv_cache_append(k, v, k_cache, v_cache, self.table, self.lens, cu_seqlens=cu)
        if whole:  # nothing was cached before: the keys are the prompt's own
            o, _ = gdn.gdn_attn_fwd(q, k, v, cu_seqlens=cu, output_lse=False)
        else:
            o, _ = gdn.gdn_attn_paged_fwd(q, k_cache, v_cache, self.table, self.lens,
                                          cu_seqlens=cu, output_lse=False)
        return o.reshape(B, T, AH * AD) @ p["out"]

    def run(self, x, cu=None, whole=False):
        """New tokens x ``[B, T, WIDTH]`` (or packed ``[1, T, WIDTH]`` with cu_seqlens) behind
        what the caches hold; returns their outputs.  ``whole``: the caches are empty."""
        self.lens += x.shape[1] if cu is None else cu.diff()
        for (kind, p), cache in zip(self.layers, self.cache):
            y = rms(x)
            x = x + (self.attention(p, y, cache, cu, whole) if kind == "A" else self.delta(p, y, cache, cu))
        return x


def packed(seqs, device="cuda"):
    """(x ``[1, T, WIDTH]``, cu_seqlens) of a list of ``[T_i, WIDTH]``."""
    lens = torch.tensor([0] + [len(s) for s in seqs])
    return torch.cat(seqs)[None].contiguous(), lens.cumsum(0).to(device=device, dtype=torch.int32)


def main():
    lens, steps = [700, 33, 1, 256], 64
    gen = torch.Generator().manual_seed(1)
    tokens = [torch.randn((n + steps, WIDTH), generator=gen).cuda().bfloat16() for n in lens]
    stack = Stack()
    stack.allocate(len(lens), max(lens) + steps)
    stack.run(*packed([t[:n] for t, n in zip(tokens, lens)]), whole=True)

    # the decode step as a graph: states, caches and lengths are updated in place
    x = torch.zeros((len(lens), 1, WIDTH), dtype=torch.bfloat16, device="cuda")
    saved = [[c.clone() for c in cache] for cache in stack.cache], stack.lens.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        stack.run(x)  # once before the capture, then back to the prompts' states
    torch.cuda.current_stream().wait_stream(stream)
    for cache, old in zip(stack.cache, saved[0]):
        for c, o in zip(cache, old):
            c.copy_(o)
    stack.lens.copy_(saved[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = stack.run(x)

    out = []
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for i in range(steps):
        x.copy_(torch.stack([t[n + i] for t, n in zip(tokens, lens)])[:, None])
        graph.replay()
        out.append(y.clone())
    end.record()
    torch.cuda.synchronize()

    again = Stack()
    again.allocate(len(lens), max(lens) + steps)
    whole = again.run(*packed(tokens), whole=True)[0].split([len(t) for t in tokens])
    want = torch.stack([w[-steps:] for w in whole]).float()
    got = torch.cat(out, 1).float()
    print(f"{steps} steps of {len(lens)} sequences: {begin.elapsed_time(end) / steps * 1e3:.0f} us each; "
          f"against one pass over everything: {float((got - want).norm() / want.norm()):.1e} (relative)")


if __name__ == "__main__":
    main()
