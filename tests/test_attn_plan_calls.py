"""Whole calls of the attention kernels' work plan on the CPU: what the host decides about a call
(csrc/gdn_attn.cuh: blocks, workspace, the plan of equal prompts) and then, for every block, what
its warp does with the lengths (staging, the choice of a plan, the walk, units dealt whole), with
the warp's lanes gone through one after the other.  Well-formed lengths: every key that a row may
see is covered once and in order.  Malformed ones (cu_seqlens that fall back or leave their range,
lengths past the table): the sequences that are malformed by themselves are left out, nothing is
done where one begins before the end of an earlier one, and a call without a workspace never cuts a unit."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "gdn_attn.cuh"

using namespace gdn;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return false; } } while (0)

static unsigned rnd_state;
static int rnd(int lo, int hi) {  // uniform over lo..hi
  rnd_state = rnd_state * 1664525u + 1013904223u;
  return lo + (int)((rnd_state >> 8) % (unsigned)(hi - lo + 1));
}
static int kinds[6];           // calls: well formed, malformed, falling back, cut, dealt whole, without workspace
static int cut_unchecked = 0;  // units cut without a workspace if that were not looked for

using F32 = AttnShape<64, 64, 64, 2, 1, 2, 1, 16, 0, 1>;

// The call as the entry points make it; `look`: whether cu_seqlens fall back is looked for.
template <class S>
bool one(const std::vector<int32_t> &cu, const std::vector<int32_t> &kv, int T, int Ttot, int H, int HKV,
         int max_len, int gpu, bool look) {
  AttnArgs a{};
  a.cu = cu.empty() ? nullptr : cu.data();
  a.kv_lens = kv.empty() ? nullptr : kv.data();
  a.n_seqs = cu.empty() ? Ttot / T : (int)cu.size() - 1;
  a.T = T; a.Ttot = Ttot; a.H = H; a.HKV = HKV; a.max_len = max_len;
  const AttnLaunch l = attn_plan_launch<S>(a, gpu);
  CHECK(l.blocks > 0 && l.blocks <= gpu && l.rows == S::kRows);
  std::vector<AttnStaged> staged(kStaged);
  bool malformed = false;
  const int threads = rnd(1, 700);  // of a block
  for (int i = 0; i < threads; i++) malformed |= attn_stage(a, staged.data(), i, threads, true);
  std::vector<AttnChunk> chunks(threads);
  bool falls = false;
  for (int i = 0; i < threads; i++) {
    const int per = (a.n_seqs + threads - 1) / threads;
    falls |= attn_falls_back(a, i * per, (i + 1) * per, chunks[i]);
  }
  for (int i = 0; i < threads; i++) falls |= attn_falls_back(chunks.data(), i);
  if (falls && look) staged[0].nq = kNothing;
  // what the definition says
  std::vector<AttnSeq> seqs;
  bool back = false;  // a sequence begins before the end of an earlier one
  for (int n = 0; n < a.n_seqs; n++) {
    AttnSeq s{};
    s.q0 = a.cu ? cu[n] : n * T;
    const int end = a.cu ? cu[n + 1] : s.q0 + T;
    if (s.q0 >= 0 && end >= s.q0 && end <= Ttot) {
      s.nq = end - s.q0;
      s.len = a.kv_lens ? kv[n] : s.nq;
      if (s.len < 0 || s.len > (a.kv_lens ? max_len : s.nq)) s.nq = s.len = 0;
      s.past = s.len - s.nq;
    }
    for (const AttnSeq &e : seqs) back |= s.nq > 0 && e.nq > 0 && s.q0 < e.q0 + e.nq;
    seqs.push_back(s);
  }
  CHECK(back == falls && (malformed || !back));
  if (look) {
    kinds[back ? 2 : malformed ? 1 : 0]++;
    if (!l.split) kinds[5]++;
  }
  std::vector<int> upto((size_t)Ttot * H);  // tiles of a row that are done
  bool cut = false, whole = false;
  for (int b = 0; b < l.blocks; b++) {
    AttnPlan<S> plan(H, HKV, a.plan_coarse, a.plan_least);
    const AttnStart st = attn_start(a, plan, staged.data(), b, l.blocks);
    if (look) CHECK(st.total < 1u << 31);
    AttnWalk<S> walk(a, plan, st, b, l.blocks);
    whole |= plan.whole || a.plan_whole;
    AttnUnit u;
    while (walk.next(u)) {
      if (!look) {
        if (u.slot >= 0 && !l.split) cut_unchecked++;
        continue;
      }
      CHECK(l.split || u.slot == -1);  // no workspace, no pieces
      CHECK(u.slot < 2 * l.blocks && u.last < l.blocks);
      CHECK((u.slot < 0) == (u.t0 == 0 && u.t1 == u.nt));
      cut |= u.slot >= 0;
      CHECK(!back && u.seq >= 0 && u.seq < a.n_seqs);
      const AttnSeq &s = seqs[u.seq];
      CHECK(u.n_tok > 0 && u.n_tok * u.gp <= S::kRows && u.kvh == u.head0 / (H / HKV));
      CHECK(u.row0 >= s.q0 && u.row0 + u.n_tok <= s.q0 + s.nq);
      CHECK(u.len == s.len && u.pos0 == s.past + u.row0 - s.q0);
      CHECK(0 <= u.t0 && u.t0 < u.t1 && u.t1 <= u.nt && (long long)u.nt * S::kTile >= u.pos0 + u.n_tok);
      for (int t = 0; t < u.n_tok; t++)
        for (int h = 0; h < u.gp; h++) {
          int &at = upto[(size_t)(u.row0 + t) * H + u.head0 + h];
          CHECK(at == u.t0);
          at = u.t1;
        }
    }
  }
  if (!look) return true;
  kinds[3] += cut;
  kinds[4] += whole;
  if (back) return true;
  for (const AttnSeq &s : seqs)
    for (int t = 0; t < s.nq; t++)
      for (int h = 0; h < H; h++)
        CHECK((long long)upto[(size_t)(s.q0 + t) * H + h] * S::kTile >= s.past + t + 1 &&
              upto[(size_t)(s.q0 + t) * H + h] > 0);
  return true;
}

template <class S>
bool call(bool look) {
  const int hkv = rnd(1, 4), H = hkv * (rnd(1, 4) == 1 ? rnd(1, 20) : 1 << rnd(0, 3));
  const int gpu = rnd(0, 2) ? rnd(1, 40) : 152;
  const int kind = look ? rnd(0, 5) : 3;
  std::vector<int32_t> cu, kv;
  int T = rnd(1, rnd(0, 1) ? 40 : 700), Ttot;
  if (kind == 0) {  // equal sequences
    Ttot = T * rnd(1, 8);
    if (rnd(0, 1)) for (int n = 0; n < Ttot / T; n++) kv.push_back(rnd(0, 9) ? rnd(0, 1500) : rnd(-5, 1600));
    return one<S>(cu, kv, T, Ttot, H, hkv, 1500, gpu, look);
  }
  cu.push_back(0);
  const int most = rnd(0, 3) ? 12 : 70;
  for (int n = rnd(1, most); n > 0; n--) cu.push_back(cu.back() + (rnd(0, 3) ? rnd(0, rnd(0, 1) ? 5 : 5000 / most) : 0));
  Ttot = cu.back();
  if (Ttot == 0) return true;
  const int n = (int)cu.size() - 1;
  if (kind == 3)  // over and over the same tokens
    for (int i = 0; i <= n; i++) cu[i] = i & 1 ? Ttot : 0;
  if (kind == 4)  // anything
    for (int i = 0; i <= n; i++) cu[i] = rnd(-5, Ttot + 20);
  if (kind == 5)  // one entry
    cu[rnd(0, n)] = rnd(0, 1) ? rnd(-100, 2 * Ttot) : rnd(0, 1) ? INT32_MIN : INT32_MAX;
  const int max_len = rnd(1, 1500);
  if (rnd(0, 1)) for (int i = 0; i < n; i++) kv.push_back(rnd(0, 9) ? rnd(0, max_len) : rnd(-5, max_len + 5));
  return one<S>(cu, kv, Ttot, Ttot, H, hkv, max_len, gpu, look);
}

// The cases that were found first.
template <class S>
bool repeated(int times, int T, int H, int HKV, bool look) {
  std::vector<int32_t> cu;
  for (int i = 0; i < times; i++) { cu.push_back(0); cu.push_back(T); }
  return one<S>(cu, {}, T, T, H, HKV, 0, 152, look);
}

int main() {
  for (int look = 1; look >= 0; look--) {
    if (!repeated<TcShape>(3, 900, 4, 1, look) || !repeated<TcShape>(3, 600, 20, 20, look) ||
        !repeated<TcShape>(4, 1000, 8, 8, look) || !repeated<F32>(20, 120, 2, 1, look)) return 1;
    for (int trial = 0; trial < 4000; trial++) {
      rnd_state = 3u + 419u * trial;
      if (!call<TcShape>(look) || !call<F32>(look)) {
        std::printf("trial %d\n", trial);
        return 1;
      }
    }
  }
  for (int i = 0; i < 6; i++)
    if (kinds[i] < 50) { std::printf("kind %d: %d calls\n", i, kinds[i]); return 1; }
  if (cut_unchecked < 50) { std::printf("cut %d times\n", cut_unchecked); return 1; }
  // more sequences than are staged
  std::vector<int32_t> cu;
  for (int n = 0; n <= 9000; n++) cu.push_back(n / 3);
  if (!one<TcShape>(cu, {}, 3000, 3000, 2, 1, 0, 152, true)) return 1;
  cu[8000] = 10;
  cu[8001] = 3000;
  if (!one<TcShape>(cu, {}, 3000, 3000, 2, 1, 0, 152, true)) return 1;
  std::printf("ok\n");
  return 0;
}
"""


def test_calls_cover_what_is_well_formed_and_cut_nothing_without_a_workspace(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "calls.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "calls"
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
