// gdn_attn.cuh -- the work plan that the attention kernels share: how the
// score matrix of a batch of sequences is cut into units and key tiles, how
// the tiles are dealt to a fixed number of blocks, and which partial results
// have to be joined afterwards.
//
// A sequence of `nq` new tokens over `len` keys has nq * H query rows.  Rows
// that read the same key/value head are stacked: a row is (token, head) with
// `gp` heads of one token next to each other.
//  * packed: nq * G <= kPack rows (G = H / HKV): one unit per key/value head
//    holds all of them (gp = G), so a decode step reads each key once.
//  * otherwise gp is the largest power of two that divides G (at most kPack)
//    and a unit is kRows rows: kRows / gp tokens of gp heads.
// A unit covers the key tiles 0 .. nt-1 of kTile keys up to its last row's
// position.  Tiles are numbered through all units and sequences, and block i of
// the grid takes the cost range [i per, (i+1) per): equal shares whatever the
// lengths, so one long sequence next to many short ones, a causal triangle and
// a single token over a long cache all fill the GPU.  A unit cut by a range's
// border leaves partial results (unnormalised output, row maximum and sum) that
// the merge kernel joins in the order of the blocks, so results do not depend
// on timing.  The plan depends on lengths that only the device knows (no
// synchronisation), so every block computes its own range from them.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {

// Shape of a unit: rows, rows of a packed unit, keys per tile, cost of one
// tile of an unpacked unit (a packed unit's tile costs 1).
template <int ROWS, int PACK, int TILE, int WIDE>
struct AttnShape {
  static constexpr int kRows = ROWS, kPack = PACK, kTile = TILE, kWide = WIDE;
};

// Partial results of one block: two slots, one for a unit that began in an
// earlier block and one for a unit that goes on in a later one.
//   o  [slot][d/4][row] float4: unnormalised output
//   ml [slot][row] float2: row maximum (log2 units) and sum
struct AttnPart {
  float4 *o;
  float2 *ml;
};

struct AttnSeq {
  int q0, nq;   // first token row and number of new tokens
  int len;      // keys, new ones included
  int past;     // position of the first new token: len - nq, negative when
                // fewer keys than new tokens are cached
  int base;     // max(past, 0): what the plan counts tiles from
};

struct AttnUnit {
  int seq;
  int row0;     // first token row
  int n_tok;    // tokens
  int head0;    // first query head of a token's rows
  int kvh;      // key/value head
  int gp;       // heads per token
  int pos0;     // position of the first token
  int len;      // keys of the sequence
  int t0, t1;   // key tiles of this block
  int nt;       // key tiles of the unit
  int slot;     // slot of the partial result, or -1 when the unit is whole
};

// Sequence n as the kernels see it; nq = 0 when its lengths are malformed
// (`bad` is then set).
__host__ __device__ __forceinline__ AttnSeq attn_seq(const AttnArgs &a, int n, bool &bad) {
  AttnSeq s;
  int end;
  if (a.cu) {
    s.q0 = a.cu[n];
    end = a.cu[n + 1];
  } else {
    s.q0 = n * a.T;
    end = s.q0 + a.T;
  }
  bad = s.q0 < 0 || end < s.q0 || end > a.Ttot;
  s.nq = bad ? 0 : end - s.q0;
  s.len = a.kv_lens ? a.kv_lens[n] : s.nq;
  if (a.kv_lens && (s.len < 0 || s.len > a.max_len)) {
    bad = true;
    s.nq = 0;
    s.len = 0;
  }
  s.past = s.len - s.nq;
  s.base = s.past > 0 ? s.past : 0;
  return s;
}

template <class S>
struct AttnPlan {
  static constexpr int kTile = S::kTile;

  int G, HKV, gp, tok, groups;  // gp, tok: heads and tokens of an unpacked unit

  __host__ __device__ AttnPlan(int H, int hkv) {
    HKV = hkv;
    G = H / hkv;
    gp = G & -G;
    if (gp > S::kPack) gp = S::kPack;
    tok = S::kRows / gp;
    groups = H / gp;
  }
  __host__ __device__ static int tiles(int keys) {
    return keys <= kTile ? 1 : (keys + kTile - 1) / kTile;
  }
  __host__ __device__ bool packed(const AttnSeq &s) const {
    return G <= S::kPack && s.nq <= S::kPack / G;
  }
  __host__ __device__ int token_tiles(const AttnSeq &s) const { return (s.nq + tok - 1) / tok; }

  // sum over i < n of floor(i / r)
  __host__ __device__ static long long floors(long long n, long long r) {
    const long long q = n / r;
    return r * (q * (q - 1) / 2) + q * (n - q * r);
  }
  // key tiles of the first x token tiles (all of them full):
  // sum over i < x of ceil((base + (i + 1) tok) / kTile)
  __host__ __device__ long long prefix(int base, long long x) const {
    if (tok >= kTile)
      return (long long)(tok / kTile) * (x * (x + 1) / 2) +
             x * ((base + kTile - 1) / kTile);
    const long long r = kTile / tok;
    const long long a = (long long)base + kTile - 1 + tok;
    const long long b = (a % kTile) / tok;
    return x * (a / kTile) + floors(b + x, r) - floors(b, r);
  }
  // key tiles of one head group of an unpacked sequence
  __host__ __device__ long long group_tiles(const AttnSeq &s) const {
    return prefix(s.base, token_tiles(s) - 1) + tiles(s.base + s.nq);
  }
  __host__ __device__ long long cost(const AttnSeq &s) const {
    if (s.nq == 0) return 0;
    if (packed(s)) return (long long)HKV * tiles(s.base + s.nq);
    return group_tiles(s) * groups * S::kWide;
  }
  __host__ __device__ int unit_cost(const AttnSeq &s) const { return packed(s) ? 1 : S::kWide; }

  // Unit that covers cost `c` (0 <= c < cost(s)) of sequence s; returns where
  // the unit begins.  t0, t1 and slot are left to the caller.
  __host__ __device__ long long find(const AttnSeq &s, int seq, long long c, AttnUnit &u) const {
    u.seq = seq;
    u.len = s.len;
    if (packed(s)) {
      u.nt = tiles(s.base + s.nq);
      u.kvh = (int)(c / u.nt);
      u.head0 = u.kvh * G;
      u.gp = G;
      u.row0 = s.q0;
      u.n_tok = s.nq;
      u.pos0 = s.past;
      return (long long)u.kvh * u.nt;
    }
    const long long per_group = group_tiles(s);
    const long long t = c / S::kWide;
    const int group = (int)(t / per_group);
    const long long rem = t - group * per_group;
    int lo = 0, hi = token_tiles(s) - 1;  // last token tile that begins at or before rem
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix(s.base, mid) <= rem) lo = mid; else hi = mid - 1;
    }
    const int first = lo * tok;
    u.n_tok = s.nq - first < tok ? s.nq - first : tok;
    u.nt = tiles(s.base + first + u.n_tok);
    u.gp = gp;
    u.head0 = group * gp;
    u.kvh = u.head0 / G;
    u.row0 = s.q0 + first;
    u.pos0 = s.past + first;
    return (group * per_group + prefix(s.base, lo)) * S::kWide;
  }
};

// first tile of a unit (beginning at cost u0, tiles of cost w) at or after cost c
__host__ __device__ __forceinline__ int attn_cut(long long u0, int w, int nt, long long c) {
  if (c <= u0) return 0;
  const long long t = (c - u0 + w - 1) / w;
  return t < nt ? (int)t : nt;
}

// Whether the border between the ranges of blocks i - 1 and i is the first one
// that cuts unit `u` (beginning at cost u0, tiles of cost w); `last` is then
// the last block with a piece of it (block i - 1 has the first piece).
__host__ __device__ __forceinline__ bool attn_merge(long long u0, int w, int nt, int i,
                                                    long long per, int &last) {
  const int cut = attn_cut(u0, w, nt, i * per);
  if (cut == 0 || cut == nt || attn_cut(u0, w, nt, (i - 1) * per) != 0) return false;
  last = i;
  while (attn_cut(u0, w, nt, (last + 1) * per) < nt) last++;
  return true;
}

// cost of each block's range
template <class S>
__host__ __device__ __forceinline__ long long attn_per(const AttnArgs &a, long long total, int n_blocks) {
  long long per = (total + n_blocks - 1) / n_blocks;
  per += per & (S::kWide - 1);
  return per < a.min_cost ? a.min_cost : per;
}

// What a block needs to start: the cost per block and the sequence its first
// cost falls into.
struct AttnStart {
  long long per;    // cost of a block's range
  long long total;  // cost of everything
  long long seq0;   // cost at which sequence `seq` begins
  int seq;
};

// Every thread of the block calls this (it synchronises the block).  Finds the
// start of cost block * per; seq = n_seqs when the block has no work.
template <int THREADS>
struct AttnStartScratch {
  long long warp_sum[THREADS / 32];
  AttnStart out;
};
template <class S, int THREADS>
__device__ __forceinline__ AttnStart attn_start(const AttnArgs &a, const AttnPlan<S> &plan,
                                                long long block, int n_blocks,
                                                AttnStartScratch<THREADS> &scratch) {
  constexpr int kWarps = THREADS / 32;
  long long *warp_sum = scratch.warp_sum;
  AttnStart &out = scratch.out;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (a.n_seqs + THREADS - 1) / THREADS;
  const int lo = min(tid * chunk, a.n_seqs), hi = min(lo + chunk, a.n_seqs);
  long long mine = 0;
  bool any_bad = false;
  for (int n = lo; n < hi; n++) {
    bool bad;
    mine += plan.cost(attn_seq(a, n, bad));
    any_bad |= bad;
  }
  if (tid == 0 && a.cu) any_bad |= a.cu[0] != 0 || a.cu[a.n_seqs] != a.Ttot;
  if (any_bad && a.flags && block == 0) atomicOr(a.flags, kFlagBadSeqlens);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) out.seq = a.n_seqs;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const long long per = attn_per<S>(a, total, n_blocks);
  const long long c = block * per;
  if (c >= before && c < before + mine) {
    long long at = before;
    for (int n = lo; n < hi; n++) {
      bool bad;
      const long long k = plan.cost(attn_seq(a, n, bad));
      if (c < at + k) {
        out.seq = n;
        out.seq0 = at;
        break;
      }
      at += k;
    }
  }
  __syncthreads();
  AttnStart r = out;
  r.per = per;
  r.total = total;
  return r;
}

// Walks the units of one block's range, in order.  One thread (or warp, all
// lanes alike) drives it.
template <class S>
struct AttnWalk {
  const AttnArgs &a;
  const AttnPlan<S> &plan;
  AttnSeq s;
  long long at, end, seq0, seq_cost;  // next cost, end of the range, current sequence's span
  int seq, block;

  __host__ __device__ AttnWalk(const AttnArgs &a_, const AttnPlan<S> &p_, const AttnStart &st, int block_)
      : a(a_), plan(p_), block(block_) {
    seq = st.seq;
    seq0 = st.seq0;
    at = block * st.per;
    end = at + st.per < st.total ? at + st.per : st.total;
    if (seq < a.n_seqs) load();
  }
  __host__ __device__ void load() {
    bool bad;
    s = attn_seq(a, seq, bad);
    seq_cost = plan.cost(s);
  }
  __host__ __device__ bool next(AttnUnit &u) {
    while (at < end) {
      while (at >= seq0 + seq_cost) {
        seq0 += seq_cost;
        if (++seq >= a.n_seqs) return false;
        load();
      }
      const long long u0 = seq0 + plan.find(s, seq, at - seq0, u);
      const int w = plan.unit_cost(s);
      u.t0 = attn_cut(u0, w, u.nt, at);
      u.t1 = attn_cut(u0, w, u.nt, end);
      at = u0 + (long long)u.nt * w;
      if (u.t0 >= u.t1) continue;
      u.slot = u.t0 > 0 ? 2 * block : (u.t1 < u.nt ? 2 * block + 1 : -1);
      return true;
    }
    return false;
  }
};

}  // namespace gdn
