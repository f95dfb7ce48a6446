"""Calls of attention over an 8-bit cache on the CPU: what the host decides about a call
(csrc/gdn_attn8.cu: which kernels, how many blocks or warps, places for partial results) and then,
for every block or warp of the plan, what it walks through.  Every key tile that a row may see is
covered once and in order, by one of the two kernels; nothing is cut without a place; the pieces of
a cut unit are where the joining looks for them.  And the order of the loads that the tensor-core
kernel's ring of scales goes by."""
from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build

PROGRAM = r"""
#include <cstdio>
#include <map>
#include <tuple>
#include <vector>

#include "gdn_attn8.cu"

namespace gdn {
int sm_count() { return 152; }
cudaError_t allow_smem(const void *, int, std::atomic<uint64_t> &) { return cudaSuccess; }
cudaError_t launch_attn8_tc(const AttnArgs &, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_attn8_merge(const AttnArgs &, int, int, int, cudaStream_t) { return cudaSuccess; }
}  // namespace gdn
using namespace gdn;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return false; } } while (0)

static unsigned state;
static int rnd(int lo, int hi) {
  state = state * 1664525u + 1013904223u;
  return lo + (int)((state >> 8) % (unsigned)(hi - lo + 1));
}
static int seen[10];  // calls with few, many, both, a warp each, a block each of many, cut, whole, 32 rows, eight heads' (of enough units for warps, for blocks)

struct Piece { int t0, t1, nt, slot, last, me; };
using Key = std::tuple<int, int, int>;  // sequence, token row, head

// Every row's pieces, in the order of the blocks.
template <class S>
bool walk_all(const AttnArgs &a, int all, const AttnLaunch &l, std::map<Key, std::vector<Piece>> &rows, int heads_of_unit = 1) {
  std::vector<AttnStaged> staged(kStaged);
  for (int i = 0; i < 7; i++) attn_stage<S>(a, staged.data(), i, 7, true);
  for (int me = 0; me < all; me++) {
    AttnPlan<S> plan(a.H, a.HKV / heads_of_unit, a.plan_coarse, a.plan_least);
    const AttnStart st = attn_start(a, plan, staged.data(), me, all);
    AttnWalk<S> walk(a, plan, st, me, all);
    AttnUnit u;
    while (walk.next(u)) {
      CHECK(u.slot < 0 || (long long)(u.slot + 1) * S::kRows <= 2LL * l.blocks * l.rows);  // within the workspace
      // each of its heads a warp's, of at most eight rows
      CHECK(heads_of_unit == 1 || (u.gp == a.H / a.HKV * heads_of_unit && u.n_tok * u.gp <= 8 * heads_of_unit));
      CHECK(u.t0 < u.t1 && u.t1 <= u.nt && u.n_tok * u.gp <= S::kRows);
      CHECK(u.slot == -1 || (l.split && u.slot < 2 * l.blocks && me < l.blocks));
      CHECK((u.slot == -1) == (u.t0 == 0 && u.t1 == u.nt));
      for (int t = 0; t < u.n_tok; t++)
        for (int h = 0; h < u.gp; h++) rows[{u.seq, u.row0 + t, u.head0 + h}].push_back({u.t0, u.t1, u.nt, u.slot, u.last, me});
    }
  }
  return true;
}

bool one(const std::vector<int32_t> &q, const std::vector<int32_t> &kv, bool packed, int H, int HKV, int max_len, int d) {
  std::vector<int32_t> cu(1, 0);
  for (int n : q) cu.push_back(cu.back() + n);
  AttnArgs a{};
  a.cu = packed ? cu.data() : nullptr;
  a.kv_lens = kv.data();
  a.n_seqs = (int)q.size(); a.T = packed ? cu.back() : q[0]; a.Ttot = cu.back(); a.H = H; a.HKV = HKV; a.max_len = max_len;
  Attn8Launch l;
  CHECK(attn8_launch(a, d, l));
  std::map<Key, std::vector<Piece>> few, many;
  int few_tile = 128;
  if (l.has_few) {
    const int grid = l.warps ? (l.few_launch.blocks + kWarps - 1) / kWarps : l.few_launch.blocks;
    bool ok;
    if (l.teams) {
      seen[l.few_launch.split ? 9 : 4]++;
      if (l.few_launch.split) few_tile = TeamShape8::kTile;
      ok = l.few_launch.split ? walk_all<TeamShape8>(l.few, grid, l.few_launch, few, kWarps) : walk_all<Shape8<1>>(l.few, grid, l.few_launch, few);
    } else if (l.warps) {
      // the device's choice
      unsigned long long tiles = 0, seqs = 0;
      for (size_t i = 0; i < q.size(); i++)
        if (q[i] > 0 && (long long)q[i] * (H / HKV) <= l.few.few_rows) {
          tiles += AttnPlan<SoloShape8>::tiles((kv[i] > q[i] ? kv[i] - q[i] : 0) + q[i]);
          seqs++;
        }
      const bool eight = HKV % kWarps == 0, solo = !l.few_launch.split || tiles <= (eight ? kShortTeam : kShort) * seqs;
      seen[solo ? 3 : eight ? 8 : 4]++;
      if (!solo && eight) few_tile = TeamShape8::kTile;
      ok = solo ? walk_all<SoloShape8>(l.few, grid * kWarps, l.few_launch, few)
           : eight ? walk_all<TeamShape8>(l.few, grid, l.few_launch, few, kWarps)
                   : walk_all<Shape8<1>>(l.few, grid, l.few_launch, few);
    } else if (l.groups == 4) {
      seen[7]++;
      ok = walk_all<Shape8<4>>(l.few, grid, l.few_launch, few);
    } else {
      ok = walk_all<Shape8<2>>(l.few, grid, l.few_launch, few);
    }
    CHECK(ok);
  }
  if (l.has_many) CHECK(walk_all<TcShape8>(l.many, l.many_launch.blocks, l.many_launch, many));
  if (l.has_few) seen[0]++;
  if (l.has_many) seen[1]++;
  if (!few.empty() && !many.empty()) seen[2]++;
  for (int n = 0; n < a.n_seqs; n++)
    for (int t = 0; t < q[n]; t++)
      for (int h = 0; h < H; h++) {
        const Key k{n, cu[n] + t, h};
        const bool f = few.count(k), m = many.count(k);
        CHECK(f != m);
        CHECK(f == ((long long)q[n] * (H / HKV) <= l.few.few_rows));
        const std::vector<Piece> &p = f ? few[k] : many[k];
        int at = 0;
        for (size_t i = 0; i < p.size(); i++) {
          CHECK(p[i].t0 == at);
          at = p[i].t1;
          // the first piece in the odd place of its block, the others in the even ones of the next blocks
          if (p.size() == 1) CHECK(p[i].slot == -1);
          else CHECK(p[i].slot == 2 * p[i].me + (i == 0 ? 1 : 0) && p[i].me == p[0].me + (int)i);
        }
        const int past = kv[n] - q[n], last = (past > 0 ? past : 0) + t + 1;  // keys that the token sees, or tiles count to
        CHECK(at == p.back().nt && (long long)at * (f ? few_tile : 128) >= last);
        if (p.size() > 1) CHECK(p[0].last == p.back().me);
        seen[p.size() > 1 ? 5 : 6]++;
      }
  return true;
}

int main() {
  const int heads[][2] = {{1, 1}, {8, 8}, {8, 2}, {6, 2}, {16, 1}, {20, 1}, {32, 2}, {40, 1}, {64, 1}, {4, 4}, {32, 8}};
  for (int i = 0; i < 900; i++) {
    state = 77u + i;
    const auto &h = heads[rnd(0, 10)];
    const bool packed = rnd(0, 1);
    const int kind = rnd(0, 4), n = kind == 0 ? rnd(1, 3) : kind == 1 ? rnd(1, 40) : kind == 4 ? rnd(200, 700) : rnd(20, 120);
    const int T = rnd(0, 2) ? rnd(1, 4) : rnd(1, 70), longest = kind == 0 ? 9000 : kind == 4 ? (rnd(0, 1) ? 300 : 1800) : 1500;
    std::vector<int32_t> q, kv;
    for (int s = 0; s < n; s++) {
      q.push_back(!packed ? T : rnd(0, 5) == 0 ? rnd(0, T) : rnd(0, 1));
      kv.push_back(rnd(0, 3) == 0 ? rnd(0, 20) : rnd(0, longest));
    }
    if (kind == 4 && rnd(0, 1)) kv[n / 2] = 20000;
    int total = 0;
    for (int x : q) total += x;
    if (total == 0) continue;
    if (!one(q, kv, packed, h[0], h[1], 20480, rnd(0, 1) ? 64 : 128)) {
      std::printf("call %d: n %d T %d packed %d heads %d/%d\n", i, n, T, packed, h[0], h[1]);
      return 1;
    }
    if (!one(q, kv, packed, h[0], h[1], kind == 4 ? 20480 : longest + 100, 128)) return 1;
  }
  // enough units for warps, but long ones, and heads that are no multiple of eight: a block's each
  for (int n = 160; n < 400; n += 25) {
    std::vector<int32_t> q(n, 1), kv;
    for (int s = 0; s < n; s++) kv.push_back(rnd(800, 2500));
    if (!one(q, kv, false, 8, 4, 20480, 64)) return 1;
  }
  // short tables: nothing is cut, whatever the number of sequences
  for (int n = 1; n < 900; n += 37) {
    std::vector<int32_t> q(n, 1), kv;
    for (int s = 0; s < n; s++) kv.push_back(rnd(0, 1000));
    if (!one(q, kv, false, 8, 2, 1024, 64)) return 1;
  }
  for (int k = 0; k < 10; k++)
    if (seen[k] < 8) { std::printf("kind %d: %d\n", k, seen[k]); return 1; }
  std::printf("ok\n");
  return 0;
}
"""


def test_every_row_is_covered_once(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def loads(units):
    """Tiles in the order of the tensor-core kernel's loads: ("k" or "v", unit, tile).  units: (tiles,
    narrow) each.  Values of a unit's last tiles come when the next one has begun."""
    out, left = [], []  # left: values still to come, for X = 0 and 1 (a wide unit's are one tile)

    def last_values(x):
        if left and left[x] is not None and not (left[2] and x == 1):
            out.append(("v", left[3], left[x]))
        if left:
            left[x] = None

    def order():
        return left and left[1] is not None and left[0] is not None and left[1] < left[0]

    for i, (n, narrow) in enumerate(units):
        if order():
            last_values(1)
        last_values(0)
        out.append(("k", i, 0))
        last_values(1)
        if narrow:
            if n > 1:
                out.append(("k", i, 1))
            for t in range(2, n):
                out += [("v", i, t - 2), ("k", i, t)]
            odd = (n - 1) & 1
            left = [n - 1 - odd, n - 2 + odd if n > 1 else None, False, i]
        else:
            for t in range(n - 1):
                out += [("v", i, t), ("k", i, t + 1)]
            left = [n - 1, n - 1, True, i]
    if order():
        last_values(1)
    last_values(0)
    last_values(1)
    return out


@pytest.mark.parametrize("stages, slots", [(5, 4), (10, 8)])  # heads of 128 and 64
def test_scales_are_read_before_their_slot_is_filled_again(stages, slots):
    """With key tile c come its scales and those of its values, into slot c % slots.  Values follow in
    the keys' order, and the loader fills position p only when position p - stages has been used: so
    the values of key tile c have to lie at or before position (key tile c + slots) - stages."""
    rng = random.Random(1)
    closest = 99
    for _ in range(3000):
        units = [(rng.choice((1, 1, 2, 2, 3, 4, 5, rng.randint(1, 30))), rng.random() < 0.5) for _ in range(rng.randint(1, 12))]
        order = loads(units)
        keys = [p for p, x in enumerate(order) if x[0] == "k"]
        values = [p for p, x in enumerate(order) if x[0] == "v"]
        assert len(keys) == len(values) == sum(n for n, _ in units)
        assert [order[p][1:] for p in keys] == [order[p][1:] for p in values]  # the same order
        for c in range(len(keys) - slots):
            closest = min(closest, keys[c + slots] - stages - values[c])
    assert closest >= 0
    # one slot less would not do (heads of 128)
    if stages == 5:
        bad = 99
        for n in (6, 7):
            order = loads([(n, True), (n, True)])
            keys = [p for p, x in enumerate(order) if x[0] == "k"]
            values = [p for p, x in enumerate(order) if x[0] == "v"]
            bad = min(bad, *(keys[c + slots - 1] - stages - values[c] for c in range(len(keys) - slots + 1)))
        assert bad < 0
