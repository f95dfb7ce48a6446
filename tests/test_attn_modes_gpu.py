"""GPU parity of bf16 attention over prompts in every mode of the work plan: grains, equal shares,
units dealt whole (equal prompts; packed ones, up to 32 of them), with several units of more than
128 rows in a row in a block.  A test without a GPU asks the plan, compiled for the host, which mode
each shape takes on a GPU of 152 processors.

The definition in 64 bits runs on the GPU here, a sequence at a time.  Tolerances as derived in
test_attn_gpu.py: with A = sum_j w_j |v_j| and S = max_j scale sum_i |q_i k_ji|,
|d o| <= 2^-8 (A + |o|) 1.01 + (2^-17 S + 2^-17) A, |d lse| <= 2^-18 S + 2^-20 |lse| + 1e-6, and a
relative error of at most 3.2e-3 over a whole result."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest
import torch

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build
from chunkwise_gated_delta_gdn_gb300 import gdn


def mixed(n, long):
    """n lengths: empty ones, single tokens, a few tokens, and long ones of odd lengths."""
    return [(0, 1, 5, long - 7 * i, 1, 130, long // 3)[i % 7] for i in range(1, n + 1)]


# name: (lengths, packed, H, HKV, d, mode, units of more than 128 rows of one block, at least)
SHAPES = {
    "equal_whole": ([700] * 4, False, 32, 32, 64, "whole", 2),
    "equal_whole_grouped": ([1025] * 3, False, 48, 12, 128, "whole", 2),
    "equal_whole_groups_of_5": ([777] * 4, False, 20, 4, 128, "whole", 2),
    "equal_whole_few_units": ([4096], False, 16, 2, 64, "whole", 2),
    "equal_grains": ([700] * 2, False, 8, 4, 128, "grains", 1),
    "equal_cut": ([3333], False, 8, 8, 64, "shares", 2),
    "packed_whole_1": ([3001], True, 32, 8, 128, "whole", 3),
    "packed_whole_31": (mixed(31, 900), True, 32, 4, 64, "whole", 2),
    "packed_whole_32": (mixed(32, 800), True, 20, 20, 128, "whole", 2),
    "packed_33": (mixed(33, 800), True, 20, 20, 128, "shares", 2),
    "packed_cut": ([3500, 0, 1, 2000], True, 4, 4, 128, "shares", 1),
}

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "gdn_attn.cuh"
using namespace gdn;
int main() {
  int n, packed, H, HKV;
  while (std::scanf("%d %d %d %d", &n, &packed, &H, &HKV) == 4) {
    std::vector<int32_t> cu(1, 0);
    int T = 0;
    for (int i = 0; i < n; i++) {
      if (std::scanf("%d", &T) != 1) return 1;
      cu.push_back(cu.back() + T);
    }
    AttnArgs a{};
    a.cu = packed ? cu.data() : nullptr;
    a.n_seqs = n; a.T = packed ? cu.back() : T; a.Ttot = cu.back(); a.H = H; a.HKV = HKV;
    const AttnLaunch l = attn_plan_launch<TcShape>(a, 152);
    std::vector<AttnStaged> staged(kStaged);
    attn_stage(a, staged.data(), 0, 1, true);
    bool whole = false, grains = false;
    int most = 0;
    for (int b = 0; b < l.blocks; b++) {
      AttnPlan<TcShape> plan(H, HKV, a.plan_coarse, a.plan_least);
      const AttnStart st = attn_start(a, plan, staged.data(), b, l.blocks);
      AttnWalk<TcShape> walk(a, plan, st, b, l.blocks);
      whole = plan.whole || a.plan_whole;
      grains = plan.over == 0;
      AttnUnit u;
      int wide = 0;
      while (walk.next(u)) wide += u.n_tok * u.gp > 128;
      most = wide > most ? wide : most;
    }
    std::printf("%s %d\n", whole ? "whole" : grains ? "grains" : "shares", most);
  }
  return 0;
}
"""


def test_shapes_take_the_modes_they_are_for(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "modes.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "modes"
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    lines = [" ".join(map(str, (len(lens), int(packed), H, HKV, *lens))) for lens, packed, H, HKV, *_ in SHAPES.values()]
    r = subprocess.run([str(exe)], input="\n".join(lines), capture_output=True, text=True, check=True)
    for (name, shape), line in zip(SHAPES.items(), r.stdout.splitlines(), strict=True):
        mode, wide = line.split()
        assert mode == shape[5] and int(wide) >= shape[6], (name, line)


def definition(q, k, v, scale):
    """(o, lse, A, S) of one sequence's last tokens, q [T, H, d], k and v [L, HKV, d], in 64 bits."""
    G = q.shape[1] // k.shape[1]
    q, k, v = (x.double().transpose(0, 1) for x in (q, k, v))
    out = []
    for h in range(q.shape[0]):  # a head at a time: scores of T x L
        kh, vh = k[h // G], v[h // G]
        s = (q[h] @ kh.T) * scale
        hidden = torch.ones_like(s, dtype=torch.bool).triu(1 + k.shape[1] - q.shape[1])
        s.masked_fill_(hidden, -torch.inf)
        lse = s.logsumexp(-1)
        w = (s - lse[:, None]).exp()
        spread = ((q[h].abs() @ kh.abs().T) * scale).masked_fill_(hidden, 0).amax(-1)
        out.append((w @ vh, lse, w @ vh.abs(), spread))
    return [torch.stack(x, 1) for x in zip(*out)]


@pytest.mark.gpu
@pytest.mark.parametrize("name", SHAPES)
def test_against_the_definition(name):
    lens, packed, H, HKV, d, *_ = SHAPES[name]
    gen = torch.Generator(device="cuda").manual_seed(len(name))
    T = sum(lens)
    q, k, v = (torch.randn((T, h, d), generator=gen, device="cuda") * std for h, std in ((H, 2.0), (HKV, 1.0), (HKV, 1.0)))
    q, k, v = (x.bfloat16() for x in (q, k, v))
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda() if packed else None
    B = 1 if packed else len(lens)
    o = torch.full((B, T // B, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T // B, H), float("nan"), device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [x.view(B, T // B, *x.shape[1:]) for x in (q, k, v)]
    gdn.gdn_attn_fwd(*args, cu_seqlens=cu, o=o, lse=lse, flags=flags)
    again = gdn.gdn_attn_fwd(*args, cu_seqlens=cu)
    assert gdn.gdn_read_device_flags(flags) == 0
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    compare(o, lse, q, [k[i:i + n] for i, n in zip(starts(lens), lens)], [v[i:i + n] for i, n in zip(starts(lens), lens)], lens)


def starts(lens):
    return [sum(lens[:i]) for i in range(len(lens))]


def compare(o, lse, q, ks, vs, q_lens):
    """o, lse of tokens q [T, H, d] against the definition over each sequence's keys and values."""
    o, lse, d = o.view(q.shape).double(), lse.view(q.shape[:2]).double(), q.shape[2]
    err = norm = 0.0
    for at, n, k, v in zip(starts(q_lens), q_lens, ks, vs):
        if n == 0:
            continue
        rows = slice(at, at + n)
        ref, ref_lse, A, S = definition(q[rows], k, v, d ** -0.5)
        diff = (o[rows] - ref).abs()
        bound = 2.0 ** -8 * 1.01 * (A + ref.abs()) + (2.0 ** -17 * S[..., None] + 2.0 ** -17) * A
        assert (diff <= bound).all(), (n, float((diff / bound).max()))
        d_lse = (lse[rows] - ref_lse).abs()
        assert (d_lse <= 2.0 ** -18 * S + 2.0 ** -20 * ref_lse.abs() + 1e-6).all(), (n, float(d_lse.max()))
        err, norm = err + float(diff.pow(2).sum()), norm + float(ref.pow(2).sum())
    assert (err / norm) ** 0.5 <= 3.2e-3, (err / norm) ** 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("H, HKV, d, page", [(16, 16, 64, 16), (16, 16, 128, 48), (30, 6, 128, 64)])
def test_long_chunks_over_a_cache(H, HKV, d, page):
    """Chunks of several units of more than 128 rows for each block, next to short ones and single
    tokens, over a cache whose pages lie about."""
    q_lens, kv_lens = [700, 1, 1205, 3, 260], [2001, 500, 1205, 901, 3333]
    gen = torch.Generator(device="cuda").manual_seed(d)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()

    q = normal(sum(q_lens), H, d, std=2.0)
    ks, vs = ([normal(n, HKV, d) for n in kv_lens] for _ in range(2))
    held = [-(-n // page) for n in kv_lens]
    order = torch.randperm(sum(held), generator=gen, device="cuda").int()
    table = torch.zeros((len(held), max(held)), dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((sum(held), page, HKV, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, n in enumerate(held):
        table[i, :n] = order[sum(held[:i]):sum(held[:i + 1])]
    lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    cu_kv = torch.tensor([0] + kv_lens).cumsum(0).int().cuda()
    gdn.gdn_kv_cache_append(torch.cat(ks)[None], torch.cat(vs)[None], kc, vc, table, lens, cu_seqlens=cu_kv)
    cu = torch.tensor([0] + q_lens).cumsum(0).int().cuda()
    o, lse = gdn.gdn_attn_paged_fwd(q[None], kc, vc, table, lens, cu_seqlens=cu)
    compare(o, lse, q, ks, vs, q_lens)
