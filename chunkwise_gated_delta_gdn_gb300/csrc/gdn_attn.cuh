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
// position.  Its tiles are grouped into grains of 2^shift tiles; every unit
// costs `over` plus its grains times a weight (both differ between packed and
// unpacked units), costs are numbered through all units and sequences, and block
// i of the grid takes the range [i per, (i+1) per).
//  * A call with little work takes the smallest grain at which there are no
//    more grains than blocks, and each block one grain: nothing waits behind
//    another unit, and no piece is smaller than 2^kMinGrain tiles.
//  * Otherwise grains are single tiles and ranges equal shares of the cost,
//    whatever the lengths: one long sequence next to many short ones and a
//    causal triangle fill the GPU alike.
//  * bf16 prompts with enough units (equal ones, or up to 32 packed) are dealt
//    whole, the longest first, to the blocks back and forth: two rounds in a row
//    add up to about the same for all, and the last, unpaired one is of the
//    shortest.  Cutting and joining costs about 16 us (kCut), so a longest block
//    that takes up to that much more than an equal share is no loss: four prompts
//    of 2048 tokens took 145 us cut, 124 whole; 16 of 512 tokens 87 and 64; one of
//    4096 tokens, 16 heads (1.7 units for each block) 80 and 63; one of 16384, 4
//    heads (1.7, the longest 520 of a share of 448) 209 and 220, and stays cut; 12001
//    packed tokens 409 and 386.  Packed prompts ask for two units for each block
//    (with one: 1 of 4096 tokens, 16 heads 80 cut, 66 whole; 6 of 400 tokens 32 and
//    26; 2 of 3000, 8 heads of 64 47 and 48) and for at most 32 sequences, a lane of
//    the plan's warp each (the same work with empty sequences up to 33, so cut: 32 of
//    512 tokens 158 us for 130, 32 of 200 73 for 59, 32 of 100 to 1500 312 for 255, 32
//    of 2048 alike).  In fp32 shares come out as fast or faster (10 x 2199
//    tokens 1100 and 1108 us).  The units of a decode step are too much alike.
// A unit cut by a range's border leaves partial results (unnormalised output,
// row maximum and sum) that the merge kernel joins in the order of the blocks,
// so results do not depend on timing.  The plan depends on lengths that only
// the device knows (no synchronisation), so every block computes it by itself.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {

// Two fp32 values in one 64-bit register pair: one instruction for both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Shape of a unit: rows, rows of a packed unit, keys per tile; cost of one tile
// of a unit and of its start and end; the same of a packed one of at most `FEW`
// rows; log2 of the smallest grain of a small call, and of the tiles up to which
// a small call's units stay whole (then it needs no workspace and no joining);
// what cutting and joining costs a block (0: prompts are not dealt whole).
template <int ROWS, int PACK, int TILE, int WIDE, int OVER, int NARROW = 1, int PACKED_OVER = OVER / 2,
          int FEW = PACK, int MIN_GRAIN = 3, int WHOLE = MIN_GRAIN, int CUT = 0>
struct AttnShape {
  static constexpr int kRows = ROWS, kPack = PACK, kTile = TILE, kFew = FEW;
  static constexpr int kMinGrain = MIN_GRAIN, kWhole = WHOLE, kCut = CUT;
  static constexpr int kWide = WIDE, kOver = OVER, kNarrow = NARROW, kPackedOver = PACKED_OVER;
  // sequences: all; 1: with at most AttnArgs::few_rows rows for a key/value head; 2: with more
  static constexpr int kOnly = 0;
  // tiles more than an equal share that a grain may have: they cost less than a second
  // unit's start and end
  static constexpr int kSlack = 4;
};
// The bf16 kernel's (gdn_attn_tc.cu).  A packed unit's tile takes 3/4 of an
// unpacked one's: 1/2, 2/3, 3/4 and 1 gave 129, 107, 104 and 109 us for two
// chunks of up to 500 tokens among 14 single ones (32 heads of 64), and 164, 153,
// 151, 189 for one of up to 1000 among 63 (heads of 128).  A unit's start and end
// take two tiles.  An unpacked one's as 0, 1, 2, 4 tiles: four prompts of 2048
// tokens 295, 160, 152, 160 us, packed prompts 663, 488, 422, 424; a packed one's
// as 0, 2, 4, 8: 256 sequences of one token 443, 410, 422, 432.
// Smallest grains of 4, 8 and 16 tiles were alike in all cases measured: below
// that a piece's start and the joining outweigh its tiles.
using TcShape = AttnShape<256, 128, 128, 4, 8, 3, 6, 128, 3, 3, 40>;
// Over a cache in 8 bits two kernels share a call's sequences: few rows go to that of
// gdn_attn8.cu, more to the bf16 one's over such a cache.
template <int ROWS>
struct FewShape8 : AttnShape<ROWS, ROWS, 128, 2, 4, 2, 4, ROWS, 1, 3> {
  static constexpr int kOnly = 1;
};
// where a unit is one warp's
struct SoloShape8 : AttnShape<16, 16, 128, 4, 2, 4, 2, 16, 1, 3> {
  static constexpr int kOnly = 1;
};
// where a unit is eight heads', each a warp's: to the plan one head with eight times the rows.
// Tiles are half as long, since they are eight times as much work for a block (256 sequences
// of up to 4096 keys 198 us with 128 keys, 194 so); an unequal share costs more than a
// second piece.
struct TeamShape8 : AttnShape<64, 64, 64, 2, 2, 2, 2, 64, 1, 3> {
  static constexpr int kOnly = 1;
  static constexpr int kSlack = 0;
};
struct TcShape8 : TcShape {
  static constexpr int kOnly = 2;
};
constexpr int kMaxGrain = 6;   // log2 of the largest one that is tried
constexpr float kBf16Inf = 0x1.ffp127f;  // what rounds to infinity in bf16

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
  int last;     // last block with a piece of the unit
};

// What the merge kernel does for block b: join the pieces of the unit that
// block b began and did not end.  Pieces: slot 2 b + 1, then slots 2 i for
// i = b + 1 .. last.
struct AttnJob {
  int row0, rows, gp, head0;  // rows = 0: nothing to do
  int last;
  int pad[3];
};
static_assert(sizeof(AttnJob) == kAttnJobBytes, "a job's place in the workspace");
__host__ __device__ __forceinline__ AttnJob attn_job(const AttnUnit &u) {
  return AttnJob{u.row0, u.n_tok * u.gp, u.gp, u.head0, u.last, {0, 0, 0}};
}

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

// The same as a kernel with shape S sees it: nq = 0 also where another one has it.
template <class S>
__host__ __device__ __forceinline__ AttnSeq attn_seq_of(const AttnArgs &a, int n, bool &bad) {
  AttnSeq s = attn_seq(a, n, bad);
  if constexpr (S::kOnly != 0) {
    const bool few = (long long)s.nq * (a.H / a.HKV) <= a.few_rows;
    if (few != (S::kOnly == 1)) s.nq = 0;
  }
  return s;
}

// Costs are counted in 32 bits: the host picks the grain of equal shares so
// that everything costs less than 2^31 (single tiles, but for prompts beyond a
// million tokens).  The plan is on the way of every call's first load, where
// 64-bit products and divisions showed.
using AttnCost = uint32_t;

template <class S>
struct AttnPlan {
  int G, HKV, groups;
  int gp, tok_log;     // heads and log2 of the tokens of an unpacked unit
  int coarse;          // log2 of the grain of equal shares
  int least;           // log2 of the smallest other one
  int shift;           // log2 of the grain, in tiles
  int wide, over;      // cost of an unpacked unit's grain, and of the unit
  int narrow, packed_over;  // of a packed one
  AttnCost per;        // cost of a block's range
  bool whole = false;  // packed prompts' units are dealt whole

  __host__ __device__ AttnPlan(int H, int hkv, int coarse_, int least_ = S::kMinGrain) {
    HKV = hkv;
    G = H / hkv;
    gp = G & -G;
    if (gp > S::kPack) gp = S::kPack;
    tok_log = 0;
    while ((gp << tok_log) < S::kRows) tok_log++;
    groups = H / gp;
    coarse = coarse_;
    least = least_;
    stream(1);
  }
  // equal shares of single tiles / one grain per block
  __host__ __device__ void stream(AttnCost p) {
    shift = coarse;
    wide = S::kWide;
    over = S::kOver;
    narrow = S::kNarrow;
    packed_over = S::kPackedOver;
    per = p;
  }
  __host__ __device__ void grains(int log) {
    shift = log;
    wide = narrow = 1;
    over = packed_over = 0;
    per = 1;
  }

  __host__ __device__ bool packed(int nq) const {
    return G <= S::kPack && nq <= S::kPack && nq * G <= S::kPack;
  }
  __host__ __device__ int token_tiles(int nq) const { return (nq + (1 << tok_log) - 1) >> tok_log; }
  __host__ __device__ static int tiles(int keys) {
    return keys <= S::kTile ? 1 : (int)(((unsigned)keys + S::kTile - 1) / S::kTile);
  }
  __host__ __device__ int grains_of(int keys) const {
    return (tiles(keys) + (1 << shift) - 1) >> shift;
  }
  __host__ __device__ static constexpr int tile_log() { return S::kTile == 128 ? 7 : 6; }
  static_assert(S::kTile == 128 || S::kTile == 64, "tile_log()");
  // sum over i < n of floor(i / 2^r)
  __host__ __device__ static AttnCost floors(AttnCost n, int r) {
    const AttnCost q = n >> r;
    return ((q * (q - 1) / 2) << r) + q * (n - (q << r));
  }
  // grains of the first x token tiles (all of them full):
  // sum over i < x of ceil((base + (i + 1) tok) / grain)
  __host__ __device__ AttnCost prefix(int base, AttnCost x) const {
    const int grain_log = tile_log() + shift;
    const AttnCost up = (1u << grain_log) - 1;
    if (tok_log > grain_log)
      return ((x * (x + 1) / 2) << (tok_log - grain_log)) + x * ((base + up) >> grain_log);
    const int r = grain_log - tok_log;
    const AttnCost a = base + up + (1u << tok_log);
    const AttnCost b = (a & up) >> tok_log;
    return x * (a >> grain_log) + floors(b + x, r) - floors(b, r);
  }
  // a sequence whose units have few rows to work on and to write
  __host__ __device__ bool few(int nq) const { return packed(nq) && nq * G <= S::kFew; }
  __host__ __device__ AttnCost own_cost(int nq) const { return few(nq) ? packed_over : over; }
  __host__ __device__ AttnCost weight(int nq) const { return few(nq) ? narrow : wide; }
  // cost of one head group of an unpacked sequence
  __host__ __device__ AttnCost group_cost(int nq, int base) const {
    const int n = token_tiles(nq);
    return (prefix(base, n - 1) + grains_of(base + nq)) * wide + (AttnCost)n * over;
  }
  __host__ __device__ AttnCost cost(int nq, int base) const {
    if (nq == 0) return 0;
    if (packed(nq)) return (AttnCost)HKV * (grains_of(base + nq) * weight(nq) + own_cost(nq));
    return group_cost(nq, base) * groups;
  }

  // Unit that covers cost `c` (0 <= c < cost) of sequence s; returns where the
  // unit begins.  t0, t1, slot and last are left to the caller.
  __host__ __device__ AttnCost find(const AttnSeq &s, int seq, AttnCost c, AttnUnit &u) const {
    u.seq = seq;
    u.len = s.len;
    if (packed(s.nq)) {
      const AttnCost each = grains_of(s.base + s.nq) * weight(s.nq) + own_cost(s.nq);
      u.nt = tiles(s.base + s.nq);
      u.kvh = (int)(c / each);
      u.head0 = u.kvh * G;
      u.gp = G;
      u.row0 = s.q0;
      u.n_tok = s.nq;
      u.pos0 = s.past;
      return u.kvh * each;
    }
    const AttnCost per_group = group_cost(s.nq, s.base);
    const int group = (int)(c / per_group);
    const AttnCost rem = c - group * per_group;
    // last token tile that begins at or before rem
    int lo = 0, hi = rem == 0 ? 0 : token_tiles(s.nq) - 1;
    AttnCost at = 0;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      const AttnCost here = prefix(s.base, mid) * wide + (AttnCost)mid * over;
      if (here <= rem) {
        lo = mid;
        at = here;
      } else {
        hi = mid - 1;
      }
    }
    place(s, group, lo, u);
    return group * per_group + at;
  }
  // token tiles of an unpacked sequence with less than t key tiles
  __host__ __device__ int shorter(int nq, int base, int t) const {
    const int n = token_tiles(nq), room = (t - 1) * S::kTile - base;
    if (nq <= room) return n;
    return room <= 0 ? 0 : (room >> tok_log < n - 1 ? room >> tok_log : n - 1);
  }
  // units of a sequence with t key tiles or more
  __host__ __device__ int units_from(int nq, int base, int t) const {
    if (nq == 0) return 0;
    if (packed(nq)) return tiles(base + nq) >= t ? HKV : 0;
    return (token_tiles(nq) - shorter(nq, base, t)) * groups;
  }
  // unit r of those of sequence s with t key tiles
  __host__ __device__ void pick(const AttnSeq &s, int t, int r, AttnUnit &u) const {
    if (!packed(s.nq)) return place(s, r % groups, shorter(s.nq, s.base, t) + r / groups, u);
    u.nt = t;
    u.kvh = r;
    u.head0 = r * G;
    u.gp = G;
    u.row0 = s.q0;
    u.n_tok = s.nq;
    u.pos0 = s.past;
  }
  // token tile `tile` of head group `group` of an unpacked sequence
  __host__ __device__ void place(const AttnSeq &s, int group, int tile, AttnUnit &u) const {
    const int first = tile << tok_log;
    u.n_tok = s.nq - first < (1 << tok_log) ? s.nq - first : 1 << tok_log;
    u.nt = tiles(s.base + first + u.n_tok);
    u.gp = gp;
    u.head0 = group * gp;
    u.kvh = u.head0 / G;
    u.row0 = s.q0 + first;
    u.pos0 = s.past + first;
  }
  // the unit behind u in the same sequence; false when u is the last one
  __host__ __device__ bool after(const AttnSeq &s, AttnUnit &u) const {
    if (packed(s.nq)) {
      u.kvh++;
      u.head0 += G;
      return u.kvh < HKV;
    }
    int tile = ((u.row0 - s.q0) >> tok_log) + 1, group = u.head0 / gp;
    if (tile == token_tiles(s.nq)) {
      tile = 0;
      if (++group == groups) return false;
    }
    place(s, group, tile, u);
    return true;
  }
  // cost of unit u
  __host__ __device__ AttnCost unit_cost(const AttnSeq &s, const AttnUnit &u) const {
    return own_cost(s.nq) + (AttnCost)((u.nt + (1 << shift) - 1) >> shift) * weight(s.nq);
  }
  // first tile at or after cost c of a unit that begins at cost u0
  __host__ __device__ int cut(const AttnSeq &s, AttnCost u0, int nt, AttnCost c) const {
    u0 += own_cost(s.nq);
    if (c <= u0) return 0;
    c -= u0;
    // by constants: a call waits for this
    const AttnCost grain = wide == 1 ? c
                           : few(s.nq) ? (c + S::kNarrow - 1) / S::kNarrow
                                          : (c + S::kWide - 1) / S::kWide;
    return grain < (AttnCost)((nt + (1 << shift) - 1) >> shift) ? (int)(grain << shift) : nt;
  }
  // last block with a piece of the unit that begins at cost u0
  __host__ __device__ int last_block(const AttnSeq &s, AttnCost u0, int nt) const {
    const AttnCost grains = (nt + (1 << shift) - 1) >> shift;
    return (int)((u0 + own_cost(s.nq) + (grains - 1) * weight(s.nq)) / per);
  }

  // Chooses; `total()` is the cost of everything under the plan as it stands.
  // Returns it for the plan that was chosen.
  template <class F>
  __host__ __device__ AttnCost choose(int n_blocks, F total) {
    AttnCost weighted = 0, share = 0;
    int log = least - 1;
    stream(1);
    while (true) {
      const AttnCost t = total();
      if (log < least) {
        weighted = t;
        share = (t + n_blocks - 1) / n_blocks;
        log = least;
      } else if (t <= (AttnCost)n_blocks) {
        return t;
      } else {
        log++;
      }
      while (log <= kMaxGrain && (2u << log) < share / S::kWide) log++;  // far too many grains
      if (log > kMaxGrain || (log > least && (1u << log) > share / S::kNarrow + S::kSlack)) break;
      grains(log);
    }
    stream(share < S::kWide ? S::kWide : share);
    return weighted;
  }
};

// The 32 lanes of the warp that makes the plan; `f(lane)` is what a lane has.  In
// a kernel this thread is one of them; on the host, where the plan is tested, they
// are gone through in order.
struct AttnLanes {
#ifdef __CUDA_ARCH__
  static constexpr int kHere = 1;  // lanes whose values a thread keeps
#else
  static constexpr int kHere = 32;
#endif
  // calls f(lane, place of its values among those kept here)
  template <class F>
  __host__ __device__ static void each(F f) {
#ifdef __CUDA_ARCH__
    f((int)(threadIdx.x & 31), 0);
#else
    for (int lane = 0; lane < 32; lane++) f(lane, lane);
#endif
  }
  template <class F>
  __host__ __device__ static uint32_t sum(F f) {
#ifdef __CUDA_ARCH__
    return __reduce_add_sync(0xffffffffu, (uint32_t)f((int)(threadIdx.x & 31)));
#else
    uint32_t r = 0;
    for (int lane = 0; lane < 32; lane++) r += f(lane);
    return r;
#endif
  }
  template <class F>
  __host__ __device__ static uint32_t max(F f) {
#ifdef __CUDA_ARCH__
    return __reduce_max_sync(0xffffffffu, (uint32_t)f((int)(threadIdx.x & 31)));
#else
    uint32_t r = 0;
    for (int lane = 0; lane < 32; lane++) {
      const uint32_t x = f(lane);
      r = x > r ? x : r;
    }
    return r;
#endif
  }
  // The lane that x falls into when their values are laid end to end, -1 when it
  // is past them; `before`: the values before that lane, or all of them.
  template <class F>
  __host__ __device__ static int holder(F f, uint32_t x, uint32_t &before) {
#ifdef __CUDA_ARCH__
    const int lane = threadIdx.x & 31;
    const uint32_t mine = f(lane);
    uint32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, x >= incl - mine && x < incl);
    const int who = hit ? __ffs(hit) - 1 : -1;
    before = __shfl_sync(0xffffffffu, hit ? incl - mine : incl, hit ? who : 31);
    return who;
#else
    before = 0;
    for (int lane = 0; lane < 32; lane++) {
      const uint32_t mine = f(lane);
      if (x < before + mine) return lane;
      before += mine;
    }
    return -1;
#endif
  }
};

// What a block needs to start: the cost of everything and the sequence its
// first cost falls into.
struct AttnStart {
  AttnCost total;
  AttnCost seq0;    // cost at which sequence `seq` begins
  int seq;          // n_seqs when the block has no work
};

// What the cost of a sequence goes by, in shared memory for the first
// kStaged sequences.
constexpr int kStaged = 4096;
struct AttnStaged {
  int nq, base;
};
// Thread `first` of `step` of a block (which then synchronise); returns whether it
// has seen malformed lengths.  `all`: look at every sequence's also where nothing
// but the flag depends on them.
template <class S = TcShape>
__host__ __device__ __forceinline__ bool attn_stage(const AttnArgs &a, AttnStaged *staged, int first,
                                                    int step, bool all) {
  bool any_bad = first == 0 && a.cu && (a.cu[0] != 0 || a.cu[a.n_seqs] != a.Ttot);
  for (int n = first; n < a.n_seqs; n += step) {
    bool bad;
    const AttnSeq s = attn_seq_of<S>(a, n, bad);
    any_bad |= bad;
    if (n < kStaged) staged[n] = AttnStaged{s.nq, s.base};
    else if (!all && !a.cu) break;
  }
  return any_bad;
}

// cu_seqlens that fall back: a sequence, as well formed as it may be by itself,
// begins before the end of an earlier one.  Together such sequences can hold more
// tokens than there are, and what the host has judged by the number of tokens does
// not hold: that costs stay below 2^31, and that nothing is cut in a call without a
// workspace.  So nothing is done then.  Looked for only where lengths are malformed,
// each thread in a chunk of the sequences, then chunk against chunk.
struct AttnChunk {
  int first, reach;  // where the first sequence with tokens begins and the last one
                     // ends; first = -1: there is none
};
constexpr int kNothing = -1;  // in the first staged sequence's nq: nothing is done
__host__ __device__ __forceinline__ bool attn_falls_back(const AttnArgs &a, int n0, int n1, AttnChunk &c) {
  c.first = -1;
  c.reach = 0;
  bool back = false, bad;
  for (int n = n0; n < n1 && n < a.n_seqs; n++) {
    const AttnSeq s = attn_seq(a, n, bad);
    if (s.nq == 0) continue;
    back |= s.q0 < c.reach;
    if (c.first < 0) c.first = s.q0;
    c.reach = s.q0 + s.nq;
  }
  return back;
}
// chunk i against the ones before it
__host__ __device__ __forceinline__ bool attn_falls_back(const AttnChunk *chunks, int i) {
  if (chunks[i].first < 0) return false;
  int before = i - 1;
  while (before >= 0 && chunks[before].first < 0) before--;
  return before >= 0 && chunks[i].first < chunks[before].reach;
}

// All THREADS threads of a block, where lengths are malformed.  Called, and with what
// it needs by value, so that it lies apart from the kernels' own code: inlined, it
// changed how that was laid out (256 sequences of one token 402 -> 405 us).
template <int THREADS>
__device__ __noinline__ void attn_stage_order(const int32_t *cu, const int32_t *kv_lens, int n_seqs,
                                              int Ttot, int max_len, AttnStaged *staged) {
  AttnArgs a{};
  a.cu = cu;
  a.kv_lens = kv_lens;
  a.n_seqs = n_seqs;
  a.Ttot = Ttot;
  a.max_len = max_len;
  AttnChunk *chunks = reinterpret_cast<AttnChunk *>(staged + kStaged);
  const int tid = threadIdx.x, per = (a.n_seqs + THREADS - 1) / THREADS;
  bool back = attn_falls_back(a, tid * per, (tid + 1) * per, chunks[tid]);
  __syncthreads();
  back |= attn_falls_back(chunks, tid);
  if (__syncthreads_or(back)) staged[0].nq = kNothing;
}
// All THREADS threads of a block, which then synchronise; block 0 reports malformed
// lengths.
template <int THREADS, class S = TcShape>
__device__ __forceinline__ void attn_stage(const AttnArgs &a, AttnStaged *staged, int block) {
  if (a.plan_total) return;
  const bool bad = attn_stage<S>(a, staged, threadIdx.x, THREADS, block == 0);
  if (bad && a.flags && block == 0) atomicOr(a.flags, kFlagBadSeqlens);
  if (__syncthreads_or(bad) && a.cu)
    attn_stage_order<THREADS>(a.cu, a.kv_lens, a.n_seqs, a.Ttot, a.max_len, staged);
}

// All lanes of one warp: choose the plan and find the start of range `block`.
template <class S>
__host__ __device__ __forceinline__ AttnStart attn_start(const AttnArgs &a, AttnPlan<S> &plan,
                                                         const AttnStaged *staged, int block,
                                                         int n_blocks) {
  AttnStart r;
  r.seq = a.n_seqs;
  r.seq0 = 0;
  if (a.plan_total) {  // equal prompts: the host has made the plan
    plan.shift = a.plan_shift;
    if (a.plan_grains) plan.grains(a.plan_shift);
    plan.per = a.plan_per;
    r.total = a.plan_total;
    const AttnCost c = block * plan.per;
    if (c < r.total) {
      r.seq = (int)(c / a.plan_seq);
      r.seq0 = r.seq * a.plan_seq;
    }
    return r;
  }
  if (staged[0].nq == kNothing) {
    r.total = 0;
    return r;
  }
  auto cost_of = [&](int n) {
    if (n < kStaged) return plan.cost(staged[n].nq, staged[n].base);
    bool bad;
    const AttnSeq s = attn_seq_of<S>(a, n, bad);
    return plan.cost(s.nq, s.base);
  };
  r.total = plan.choose(n_blocks, [&] {
    return AttnLanes::sum([&](int lane) {
      AttnCost mine = 0;
      for (int n = lane; n < a.n_seqs; n += 32) mine += cost_of(n);
      return mine;
    });
  });
  if (S::kCut != 0 && !a.kv_lens && a.n_seqs <= 32 && plan.over != 0) {
    auto nq = [&](int lane) { return lane < a.n_seqs ? staged[lane].nq : 0; };
    const int units = AttnLanes::sum([&](int lane) { return plan.units_from(nq(lane), 0, 1); });
    const AttnCost longest = AttnLanes::max([&](int lane) {
      return nq(lane) ? plan.grains_of(nq(lane)) * plan.weight(nq(lane)) + plan.own_cost(nq(lane)) : 0u;
    });
    plan.whole = units >= 2 * n_blocks && longest <= plan.per + S::kCut;
    if (plan.whole) return r;
  }
  const AttnCost c = block * plan.per;
  if (c >= r.total) return r;
  AttnCost before = 0;
  for (int n0 = 0; n0 < a.n_seqs; n0 += 32) {
    AttnCost here;
    const int who = AttnLanes::holder(
        [&](int lane) { return n0 + lane < a.n_seqs ? cost_of(n0 + lane) : 0u; }, c - before, here);
    before += here;
    if (who >= 0) {
      r.seq = n0 + who;
      r.seq0 = before;
      return r;
    }
  }
  return r;
}

// Walks the units of one block's range, in order.
template <class S>
struct AttnWalk {
  const AttnArgs &a;
  const AttnPlan<S> &plan;
  AttnSeq s;
  AttnUnit u;
  AttnCost at, end, u0;  // start and end of the range, start of the sequence or unit
  int seq, block;
  bool fresh;            // the sequence is still to be looked up
  int blocks, round;     // units dealt whole
  AttnSeq mine[AttnLanes::kHere];  // of packed prompts: lane i has sequence i

  __host__ __device__ AttnWalk(const AttnArgs &a_, const AttnPlan<S> &p_, const AttnStart &st,
                               int block_, int blocks_ = 0)
      : a(a_), plan(p_), block(block_), blocks(blocks_), round(0) {
    at = block * plan.per;
    end = at + plan.per < st.total ? at + plan.per : st.total;
    seq = st.seq;
    u0 = st.seq0;
    fresh = true;
    if (S::kCut != 0 && plan.whole)
      AttnLanes::each([&](int lane, int i) {
        bool bad;
        mine[i].nq = mine[i].base = 0;
        if (lane < a.n_seqs) mine[i] = attn_seq_of<S>(a, lane, bad);
      });
  }
  // place of this block's next unit among those that are dealt whole
  __host__ __device__ int turn() {
    const int r = round++;
    return r * blocks + (r & 1 ? blocks - 1 - block : block);
  }
  // unit i of packed prompts in order of length; all lanes of a warp
  __host__ __device__ bool deal(int i, AttnUnit &out) const {
    auto at = [&](int lane) -> const AttnSeq & { return mine[lane & (AttnLanes::kHere - 1)]; };
    auto from = [&](int t) {
      return (int)AttnLanes::sum([&](int lane) { return plan.units_from(at(lane).nq, at(lane).base, t); });
    };
    if (i >= from(1)) return false;
    int lo = 1, hi = AttnLanes::max([&](int lane) { return plan.tiles(at(lane).base + at(lane).nq); });
    while (lo < hi) {  // the most tiles that more than i units have
      const int mid = (lo + hi + 1) >> 1;
      if (from(mid) > i) lo = mid; else hi = mid - 1;
    }
    i -= from(lo + 1);
    uint32_t before;
    const int who = AttnLanes::holder(
        [&](int lane) {
          return plan.units_from(at(lane).nq, at(lane).base, lo) - plan.units_from(at(lane).nq, at(lane).base, lo + 1);
        },
        i, before);
    bool bad;
    const AttnSeq one = attn_seq_of<S>(a, who, bad);
    plan.pick(one, lo, i - (int)before, out);
    out.seq = who;
    out.len = one.len;
    return true;
  }
  __host__ __device__ bool next(AttnUnit &out) {
    if constexpr (S::kCut != 0) {
      if (plan.whole || a.plan_whole) return next_whole(out);
    }
    while (seq < a.n_seqs && u0 < end) {
      if (fresh) {
        bool bad;
        s = attn_seq_of<S>(a, seq, bad);
        if (s.nq == 0) {
          seq++;
          continue;
        }
        u0 += plan.find(s, seq, at > u0 ? at - u0 : 0, u);
        fresh = false;
      }
      out = u;
      out.t0 = plan.cut(s, u0, u.nt, at);
      out.t1 = plan.cut(s, u0, u.nt, end);
      out.slot = out.t0 > 0 ? 2 * block : (out.t1 < u.nt ? 2 * block + 1 : -1);
      out.last = out.slot == 2 * block + 1 ? plan.last_block(s, u0, u.nt) : block;
      u0 += plan.unit_cost(s, u);
      if (!plan.after(s, u)) {
        fresh = true;
        seq++;
      }
      if (out.t0 < out.t1) return true;
    }
    return false;
  }
  __host__ __device__ bool next_whole(AttnUnit &out) {
    if (plan.whole) {
      if (!deal(turn(), out)) return false;
    } else {
      const int all = a.n_seqs * plan.groups, i = turn();
      const int tile = plan.token_tiles(a.T) - 1 - i / all;
      if (tile < 0) return false;
      bool bad;
      out.seq = i % all / plan.groups;
      const AttnSeq one = attn_seq_of<S>(a, out.seq, bad);
      plan.place(one, i % plan.groups, tile, out);
      out.len = one.len;
    }
    out.t0 = 0;
    out.t1 = out.nt;
    out.slot = -1;
    out.last = block;
    return true;
  }
};

// Most units that a call can have, from what the host knows.
template <class S>
inline long long attn_most_units(const AttnArgs &a) {
  const AttnPlan<S> plan(a.H, a.HKV, 0);
  const long long groups = plan.groups > a.HKV ? plan.groups : a.HKV;
  if (!a.cu)
    return a.n_seqs * (plan.packed(a.T) ? (long long)a.HKV : (long long)plan.groups * plan.token_tiles(a.T));
  return a.n_seqs * groups + (long long)plan.groups * (a.Ttot >> plan.tok_log);
}

// Grain of equal shares for which at most `units` units of up to `longest`
// keys cost less than 2^31; -1 when there is none.
template <class S>
inline int attn_coarse(long long units, int longest) {
  for (int log = 0; log < 24; log++) {
    const long long grains = (AttnPlan<S>::tiles(longest) + (1LL << log) - 1) >> log;
    if (units <= (1LL << 31) / (grains * S::kWide + S::kOver)) return log;
  }
  return -1;
}

// The plan of equal prompts (lengths that the host knows), into `a`; returns
// whether a unit may be cut between blocks.
template <class S>
inline bool attn_plan_prompts(AttnArgs &a, int n_blocks) {
  AttnPlan<S> plan(a.H, a.HKV, a.plan_coarse, a.plan_least);
  a.plan_total = plan.choose(n_blocks, [&] { return plan.cost(a.T, 0) * a.n_seqs; });
  a.plan_seq = plan.cost(a.T, 0);
  a.plan_per = plan.per;
  a.plan_shift = plan.shift;
  a.plan_grains = plan.over == 0;
  const int all = a.n_seqs * plan.groups;
  const long long units = (long long)all * plan.token_tiles(a.T);
  a.plan_whole = S::kCut != 0 && !a.plan_grains && !plan.packed(a.T) && units >= n_blocks &&
                 units < INT32_MAX / 2;
  // the block with the most to do; with many units each they are all alike
  for (int b = 0; a.plan_whole && units < 4LL * n_blocks && b < n_blocks; b++) {
    AttnCost load = 0;
    for (int r = 0; r < 4; r++) {
      const int tile = plan.token_tiles(a.T) - 1 - (r * n_blocks + (r & 1 ? n_blocks - 1 - b : b)) / all;
      if (tile < 0) break;
      const int tokens = (tile + 1) << plan.tok_log;
      load += plan.tiles(tokens < a.T ? tokens : a.T) * plan.wide + plan.over;
    }
    a.plan_whole = load <= plan.per + S::kCut;
  }
  if (a.plan_whole) return false;
  return !(a.plan_grains && plan.tiles(a.T) <= 1 << plan.shift);
}

// The launch of a call, given the blocks that the GPU holds, and the plan where
// the host can make it, into `a`.
template <class S>
AttnLaunch attn_plan_launch(AttnArgs &a, int blocks) {
  AttnLaunch l;
  l.blocks = blocks;
  l.rows = S::kRows;
  a.plan_total = 0;
  a.plan_whole = 0;
  // Nothing is cut when every unit is short and gets a block.
  const long long units = attn_most_units<S>(a);
  // A sequence's tiles are counted to the position of its last new token as if
  // its first were at 0 or later: past its keys where it has fewer of them.
  const int tokens = a.cu ? a.Ttot : a.T;
  const int longest = a.kv_lens && a.max_len > tokens ? a.max_len : tokens;
  l.split = !(AttnPlan<S>::tiles(longest) <= 1 << S::kWhole && units <= blocks);
  a.plan_least = l.split ? S::kMinGrain : S::kWhole;
  if (!l.split) l.blocks = units < 1 ? 1 : (int)units;
  a.plan_coarse = attn_coarse<S>(units, longest);
  if (a.plan_coarse < 0) {
    l.blocks = 0;
    return l;
  }
  if (!a.cu && !a.kv_lens && a.T > 0) l.split = attn_plan_prompts<S>(a, l.blocks);
  return l;
}

}  // namespace gdn
