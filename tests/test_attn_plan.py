"""The attention kernels' work plan on the CPU: the host compiles the plan that
the kernels use (csrc/gdn_attn.cuh) into a program that deals random batches to
random numbers of blocks and checks that every key a row may see is covered
once, that pieces of a unit get distinct slots and that the merge finds exactly
them."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <tuple>
#include <vector>

#include "gdn_attn.cuh"

using namespace gdn;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return false; } } while (0)

static unsigned rnd_state;
static int grains_chosen = 0;
static int rnd(int lo, int hi) {  // uniform over lo..hi
  rnd_state = rnd_state * 1664525u + 1013904223u;
  return lo + (int)((rnd_state >> 8) % (unsigned)(hi - lo + 1));
}

template <class S>
bool one(const std::vector<int> &q, const std::vector<int> &kv, int H, int HKV, int blocks, int force, int coarse) {
  std::vector<int32_t> cu(1, 0), lens(kv.begin(), kv.end());
  for (int n : q) cu.push_back(cu.back() + n);
  AttnArgs a{};
  a.cu = cu.data(); a.kv_lens = lens.data(); a.n_seqs = (int)q.size(); a.Ttot = cu.back();
  a.H = H; a.HKV = HKV; a.max_len = 1 << 30;
  AttnPlan<S> plan(H, HKV, coarse);
  CHECK(H % plan.gp == 0 && plan.G % plan.gp == 0 && plan.gp << plan.tok_log == S::kRows);
  std::vector<long long> seq0;
  auto sum = [&] {
    AttnCost total = 0;
    bool bad;
    seq0.clear();
    for (int n = 0; n < a.n_seqs; n++) {
      seq0.push_back(total);
      const AttnSeq s = attn_seq(a, n, bad);
      total += plan.cost(s.nq, s.base);
    }
    return total;
  };
  AttnCost total = sum();
  if (force >= 0) {  // any grain and any share, not only those that the kernels choose
    plan.grains(force);
    total = sum();
    plan.per = total ? (total + blocks - 1) / blocks : 1;
  } else {
    total = plan.choose(blocks, sum);
    CHECK(sum() == total);
    grains_chosen += plan.over == 0;
  }
  const long long per = plan.per;
  CHECK(per * blocks >= total && per >= 1);
  std::map<std::pair<int, int>, std::vector<int>> seen;  // (row, head) -> tiles
  std::map<std::tuple<int, int>, std::vector<int>> pieces;  // (row0, head0) -> slots in order
  std::map<std::tuple<int, int>, AttnUnit> units;
  std::set<int> slots;
  std::vector<AttnUnit> begun;
  for (int b = 0; b < blocks; b++) {
    AttnStart st{};
    st.total = total; st.seq = a.n_seqs;
    for (int n = 0; n < a.n_seqs; n++) {
      bool bad;
      const AttnSeq s = attn_seq(a, n, bad);
      const long long c = plan.cost(s.nq, s.base);
      if (b * per >= seq0[n] && b * per < seq0[n] + c) { st.seq = n; st.seq0 = seq0[n]; }
    }
    AttnWalk<S> walk(a, plan, st, b);
    AttnUnit u;
    while (walk.next(u)) {
      CHECK(0 <= u.t0 && u.t0 < u.t1 && u.t1 <= u.nt);
      CHECK(u.n_tok > 0 && u.n_tok * u.gp <= S::kRows && u.kvh == u.head0 / plan.G);
      CHECK(u.row0 >= cu[u.seq] && u.row0 + u.n_tok <= cu[u.seq + 1]);
      CHECK(u.len == kv[u.seq] && u.pos0 == kv[u.seq] - q[u.seq] + u.row0 - cu[u.seq]);
      CHECK((long long)u.nt * S::kTile >= u.pos0 + u.n_tok);
      CHECK((u.slot < 0) == (u.t0 == 0 && u.t1 == u.nt));
      if (u.slot >= 0) {
        CHECK(u.slot / 2 == b && slots.insert(u.slot).second);
        pieces[{u.row0, u.head0}].push_back(u.slot);
        if (u.slot & 1) begun.push_back(u);
      }
      units[{u.row0, u.head0}] = u;
      for (int t = 0; t < u.n_tok; t++)
        for (int g = 0; g < u.gp; g++)
          for (int k = u.t0; k < u.t1; k++) seen[{u.row0 + t, u.head0 + g}].push_back(k);
    }
  }
  for (int n = 0; n < a.n_seqs; n++)
    for (int t = 0; t < q[n]; t++)
      for (int h = 0; h < H; h++) {
        const std::vector<int> &v = seen[{cu[n] + t, h}];
        const int visible = kv[n] - q[n] + t + 1;
        CHECK(!v.empty() && (long long)v.size() * S::kTile >= visible);
        for (size_t i = 0; i < v.size(); i++) CHECK(v[i] == (int)i);  // in order, each once
      }
  // the merge goes by what each unit's first block says of the last one
  std::set<std::tuple<int, int>> merged;
  for (const AttnUnit &u : begun) {
    CHECK(merged.insert({u.row0, u.head0}).second);
    std::vector<int> want{u.slot};
    for (int b = u.slot / 2 + 1; b <= u.last; b++) want.push_back(2 * b);
    CHECK((pieces[{u.row0, u.head0}] == want));
    const AttnJob job = attn_job(u);
    CHECK(job.rows == u.n_tok * u.gp && job.rows <= S::kRows && job.last == u.last);
  }
  CHECK(merged.size() == pieces.size());
  return true;
}

int main() {
  for (int trial = 0; trial < 600; trial++) {
    rnd_state = 7u + 977u * trial;
    const int hkv = rnd(1, 4), g = rnd(1, 4) == 1 ? rnd(1, 20) : 1 << rnd(0, 4);
    std::vector<int> q, kv;
    for (int n = rnd(1, 12); n > 0; n--) {
      const int kind = rnd(0, 5);
      const int nq = kind == 0 ? 0 : kind < 3 ? 1 : kind < 5 ? rnd(1, 40) : rnd(1, 700);
      q.push_back(nq);
      kv.push_back(rnd(0, 9) == 0 ? rnd(0, nq) : nq + rnd(0, rnd(0, 1) ? 100 : 1500));
    }
    const int blocks = rnd(0, 1) ? rnd(1, 9) : rnd(10, 200), force = rnd(0, 1) ? -1 : rnd(0, 4);
    if (!one<AttnShape<64, 64, 64, 1, 1>>(q, kv, hkv * g, hkv, blocks, force, trial % 3) ||
        !one<AttnShape<256, 128, 128, 2, 4>>(q, kv, hkv * g, hkv, blocks, force, trial % 3) ||
        !one<TcShape>(q, kv, hkv * g, hkv, blocks, force, trial % 3) ||
        !one<AttnShape<64, 64, 64, 2, 1, 2, 1, 16, 0, 1>>(q, kv, hkv * g, hkv, blocks, force, trial % 3)) {
      std::printf("trial %d: hkv %d g %d blocks %d\n", trial, hkv, g, blocks);
      return 1;
    }
  }
  if (grains_chosen < 50) { std::printf("grains chosen %d times\n", grains_chosen); return 1; }
  std::printf("ok\n");
  return 0;
}
"""


def test_plan_covers_every_visible_key_once(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "plan.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "plan"
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


WHOLE = PROGRAM[:PROGRAM.index("int main() {")] + r"""
// Calls of short units with a block for each (or more): nothing may be cut, there is no workspace.
template <class S>
bool whole(const std::vector<int> &q, const std::vector<int> &kv, int H, int HKV, int spare) {
  std::vector<int32_t> cu(1, 0), lens(kv.begin(), kv.end());
  for (int n : q) cu.push_back(cu.back() + n);
  AttnArgs a{};
  a.cu = cu.data(); a.kv_lens = lens.data(); a.n_seqs = (int)q.size(); a.Ttot = cu.back();
  a.H = H; a.HKV = HKV; a.max_len = 1 << 30;
  const int blocks = (int)attn_most_units<S>(a) + spare;
  if (blocks < 1) return true;
  AttnPlan<S> plan(H, HKV, 0, S::kWhole);
  bool bad;
  auto sum = [&] {
    AttnCost total = 0;
    for (int n = 0; n < a.n_seqs; n++) { const AttnSeq s = attn_seq(a, n, bad); total += plan.cost(s.nq, s.base); }
    return total;
  };
  const AttnCost total = plan.choose(blocks, sum);
  CHECK(plan.over == 0 && plan.per == 1 && total <= (AttnCost)blocks && 1 << plan.shift >= 1 << S::kWhole);
  for (int n = 0; n < a.n_seqs; n++) CHECK(plan.grains_of(kv[n] > q[n] ? kv[n] : q[n]) == 1);
  return true;
}
int main() {
  for (int trial = 0; trial < 3000; trial++) {
    rnd_state = 11u + 613u * trial;
    const int hkv = rnd(1, 4), g = rnd(1, 20);
    std::vector<int> q, kv;
    for (int n = rnd(1, 12); n > 0; n--) {
      q.push_back(rnd(0, rnd(0, 1) ? 3 : 128));
      kv.push_back(rnd(0, 128));
    }
    const int spare = rnd(0, 1) ? 0 : rnd(0, 100);
    if (!whole<TcShape>(q, kv, hkv * g, hkv, spare) ||
        !whole<AttnShape<64, 64, 64, 2, 1, 2, 1, 16, 0, 1>>(q, kv, hkv * g, hkv, spare)) return 1;
  }
  std::printf("ok\n");
  return 0;
}
"""


def test_short_units_with_a_block_each_stay_whole(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "whole.cu"
    src.write_text(WHOLE)
    exe = tmp_path / "whole"
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


DEAL = PROGRAM[:PROGRAM.index("int main() {")] + r"""
// Prompts whose units are dealt whole: every (row, head) in one unit with all of its keys, the
// units in order of length, and (equal prompts) every unit to one block.
template <class S>
bool covered(const std::vector<AttnUnit> &units, const std::vector<int> &q, int H, const AttnPlan<S> &plan) {
  std::set<std::pair<int, int>> rows;
  std::vector<int> at(1, 0);
  for (int n : q) at.push_back(at.back() + n);
  for (const AttnUnit &u : units) {
    CHECK(u.seq >= 0 && u.seq < (int)q.size() && u.len == q[u.seq] && u.kvh == u.head0 / plan.G);
    CHECK(u.n_tok > 0 && u.n_tok * u.gp <= S::kRows && u.row0 >= at[u.seq] && u.row0 + u.n_tok <= at[u.seq + 1]);
    CHECK(u.pos0 == u.row0 - at[u.seq] && u.nt == AttnPlan<S>::tiles(u.pos0 + u.n_tok));
    for (int t = 0; t < u.n_tok; t++)
      for (int g = 0; g < u.gp; g++) CHECK(rows.insert({u.row0 + t, u.head0 + g}).second);
  }
  CHECK((long long)rows.size() == (long long)at.back() * H);
  return true;
}
template <class S>
bool ragged(const std::vector<int> &q, int H, int HKV) {
  std::vector<int32_t> cu(1, 0);
  for (int n : q) cu.push_back(cu.back() + n);
  AttnArgs a{};
  a.cu = cu.data(); a.n_seqs = (int)q.size(); a.Ttot = cu.back(); a.H = H; a.HKV = HKV;
  const AttnPlan<S> plan(H, HKV, 0);
  auto from = [&](int t) {
    int n = 0;
    for (int x : q) n += plan.units_from(x, 0, t);
    return n;
  };
  std::vector<AttnUnit> units;
  int longest = 1 << 30;
  for (int i = 0; i < from(1); i++) {
    int t = 1;
    while (from(t + 1) > i) t++;
    int r = i - from(t + 1), who = 0;
    for (; who < (int)q.size(); who++) {
      const int have = plan.units_from(q[who], 0, t) - plan.units_from(q[who], 0, t + 1);
      if (r < have) break;
      r -= have;
    }
    CHECK(who < (int)q.size());
    bool bad;
    AttnUnit u;
    const AttnSeq s = attn_seq(a, who, bad);
    plan.pick(s, t, r, u);
    u.seq = who; u.len = s.len;
    CHECK(u.nt == t && t <= longest);
    longest = t;
    units.push_back(u);
  }
  return covered<S>(units, q, H, plan);
}
template <class S>
bool equal(int n, int T, int H, int HKV, int blocks) {
  AttnArgs a{};
  a.n_seqs = n; a.T = T; a.Ttot = n * T; a.H = H; a.HKV = HKV; a.plan_least = S::kMinGrain;
  if (attn_plan_prompts<S>(a, blocks) || !a.plan_whole) return true;
  const AttnPlan<S> plan(H, HKV, 0);
  std::vector<AttnUnit> units;
  long long most = 0, total = 0;
  for (int b = 0; b < blocks; b++) {
    AttnStart st{};
    st.seq = n;
    AttnWalk<S> walk(a, plan, st, b, blocks);
    AttnUnit u;
    long long load = 0;
    while (walk.next(u)) {
      CHECK(u.t0 == 0 && u.t1 == u.nt && u.slot == -1);
      load += u.nt;
      units.push_back(u);
    }
    most = load > most ? load : most;
    total += load;
  }
  grains_chosen++;
  // two rounds in a row differ by no more than neighbouring lengths, the last one is short
  const long long longest = plan.tiles(T);
  CHECK(most <= total / blocks + longest + (long long)units.size() / blocks + 2);
  return covered<S>(units, std::vector<int>(n, T), H, plan);
}
int main() {
  for (int trial = 0; trial < 400; trial++) {
    rnd_state = 5u + 811u * trial;
    const int hkv = rnd(1, 4), g = rnd(1, 4) == 1 ? rnd(1, 20) : 1 << rnd(0, 4);
    std::vector<int> q;
    for (int n = rnd(1, 12); n > 0; n--) q.push_back(rnd(0, 5) == 0 ? 0 : rnd(1, rnd(0, 1) ? 9 : 900));
    using F = AttnShape<64, 64, 64, 2, 1, 2, 1, 16, 0, 1, 40>;
    if (!ragged<TcShape>(q, hkv * g, hkv) || !ragged<F>(q, hkv * g, hkv)) return 1;
    const int n = rnd(1, 6), T = rnd(1, rnd(0, 1) ? 200 : 3000), blocks = rnd(1, 60);
    if (!equal<TcShape>(n, T, hkv * g, hkv, blocks) || !equal<F>(n, T, hkv * g, hkv, blocks)) return 1;
  }
  if (grains_chosen < 50) { std::printf("dealt %d times\n", grains_chosen); return 1; }
  std::printf("ok\n");
  return 0;
}
"""


def test_units_dealt_whole_cover_every_row_once(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "deal.cu"
    src.write_text(DEAL)
    exe = tmp_path / "deal"
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
