// gdn_attn8.cu -- attention of few query rows (a decode step) over a paged cache
// held in 8 bits: e4m3 values with an fp32 scale for each block of 16 tokens and
// key/value head; and the choice of kernels of a call (more rows: gdn_attn_tc.cu).
//
//   s_j = scale a_j q.k_j,  m = max_j s_j,  l = sum_j e^(s_j - m),
//   o = sum_j e^(s_j - m) b_j v_j / l,      lse = m + ln l
// with k_j, v_j the 8-bit values and a_j, b_j their blocks' scales.
//
// A decode step reads each key and value once and has 8 products for each value
// read, so memory is to be the bound, and what stands between the loads and it is
// kept small: a unit (a sequence's rows of one key/value head, at most 16 or 32) has
// eight warps, each of which takes every eighth block of 16 keys by itself, from
// copying it (cp.async into a ring of its own) to the weighted sum; nothing
// synchronises warps until a unit's end.  In larger calls a unit is eight heads', each a
// warp's, or, where there are thousands of short ones, a warp's (kShort).  With the keys as the M
// and the query rows as the N dimension of mma.sync (m16n8k16), 8 rows cost no more
// than there are:
//   S^T = K Q^T   (16 keys x 8 rows),  O^T += V^T P^T  (D x 8 rows)
// (One 128-row tile of the tcgen05 instructions would be mostly empty, and its way
// through tensor memory and barriers, 2000 clocks for 128 keys, longer than the 1400 in
// which memory brings them.)  The 8-bit values go to fp16, where they are exact,
// straight into the fragments: which of a key's elements a thread takes for which k is
// free as long as Q's fragment does the same, so a thread reads 32 bytes of a key in a
// row; V's keys are paired by byte permutes.  Scales are applied to scores and weights,
// a scalar each for the 16 keys of a step.  Q is scaled by a power of two for each row
// into the middle of fp16's range (exact but for elements below 2^-28 of the row's
// largest).
//
// Weights are rounded to fp16 for the product with V: e^(s - m) b 2^6 relative to
// the largest such product so far, moved when it is outgrown by 2^8, so they stay
// below 2^15 and what is below 2^-30 of the largest one is lost.  The sum l has a
// maximum of its own (of s alone), in fp32.
//
// 256 sequences of up to 4096 keys, 32/8 heads of 128: 186 us (1.17 GB, 6.3 TB/s), 402 over
// a bf16 cache.  64 sequences over 4096 keys, heads of 64: 55 us (4.9 TB/s): half
// the bytes for the same instructions, 57% of the issue slots.  One token over 131072
// keys, 16/2 heads: 25 us, 10 of them loads, the rest start, plan, first loads and joining.
// Three blocks to an SM, with two stages each, gave 205 for 215 us of the first and 31 for
// 25.5 of the last; four of four warps 204 for 194 and 31 for 26.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "gdn_attn.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kSlice = kScaleBlock;  // keys of a warp's step
// How a unit is shared by a block's warps: each has every eighth slice of its keys, one of
// its eight heads, or a unit of its own.
enum Share { kKeys, kHeads, kUnits };
template <int NT, Share SHARE = kKeys>
using Shape8 = std::conditional_t<SHARE == kUnits, SoloShape8, std::conditional_t<SHARE == kHeads, TeamShape8, FewShape8<NT == 4 ? 32 : 16>>>;
static_assert(Shape8<1>::kTile / kSlice == kWarps, "a slice of each tile for each warp");
// Blocks of an SM: 32 rows take 255 registers of a thread for their output alone.
template <int NT>
constexpr int blocks_per_sm() { return NT == 4 ? 1 : 2; }
constexpr float kLag = 8.f;    // log2 growth of a maximum that is let stand
constexpr float kNone = -0x1p120f;  // a maximum before any key: finite, so that -inf scores weigh 0
constexpr float kShift = 6.f;  // log2 of the weights' factor

// How many units there are: few; enough for the GPU's warps; enough for its blocks, eight
// heads at a time.
enum Units { kFewUnits, kForWarps, kForBlocks };
template <int D, int NT, bool MANY = false>
struct Smem {
  static constexpr int kSliceBytes = 2 * kSlice * D;
  static constexpr int kStages = (D == 128 ? 6 : 12) / blocks_per_sm<NT>();
  static constexpr int kCopies = MANY ? kWarps : 1;  // of Q
  static constexpr int kRow = D + 4;  // floats of a row where warps are joined
  static constexpr int kScale = kWarps * kStages * kSliceBytes;  // [warp][stage][2], behind the ring [warp][stage][keys, values]
  static constexpr int kQ = kScale + kWarps * kStages * 8;       // [nt][two k steps][lane][k step] two registers
  static constexpr int kQBytes = NT * (D / 16) * 32 * 8;
  static constexpr int kFactor = kQ + kCopies * kQBytes;         // [rows]
  // [warp][rows] maximum, sum, maximum with V's scale (where a unit is a block's, in the
  // place of a second copy of Q)
  static constexpr int kEnd = kFactor + kCopies * NT * 8 * 4, kJoinBytes = kWarps * NT * 8 * 12;
  static constexpr int kJoin = MANY ? kQ + kQBytes : kEnd;
  static constexpr int kBytes = kEnd + (MANY ? 0 : kJoinBytes);
  static_assert(!MANY || kJoinBytes <= kQBytes, "in a copy's place");
  static_assert(kWarps * NT * 8 * kRow * 4 <= kScale, "joined in the ring's place");
  static_assert(kStaged * sizeof(AttnStaged) + kThreads * sizeof(AttnChunk) <= kScale, "staging in the ring's place");
};
template <int D, int NT, bool MANY = false>
constexpr bool fits() { return blocks_per_sm<NT>() * (Smem<D, NT, MANY>::kBytes + 1024) <= 233472; }
static_assert(fits<64, 2>() && fits<128, 2>() && fits<64, 4>() && fits<128, 4>(), "shared memory of one SM");
static_assert(fits<64, 1, true>() && fits<128, 1, true>(), "shared memory of one SM");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two 8-bit values (the low or high half of x) as two fp16
__device__ __forceinline__ uint32_t half_lo(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t half_hi(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
// 16 bytes in the background, read once; zeros for those past `bytes`.  L2 fetches no
// more than 64 bytes around them: with its default, a 64-byte row came with the next
// head's, gone again before that was read (64 sequences over 4096 keys, 8 heads of 64:
// 95 us, twice the bytes; so 62.5).
__device__ __forceinline__ void copy16(uint32_t to, const void *from, uint64_t policy, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::64B [%0], [%1], 16, %2, %3;" ::"r"(to), "l"(from), "r"(bytes), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void *from, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::64B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "l"(policy) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// NT: groups of 8 rows.  SOLO: a row is one warp's, all of its keys, so that nothing
// but the plan's start is shared by a block's warps.  MANY: partial results lie as
// gdn_attn8_merge_kernel reads them.  All threads of a block, lengths staged.
template <int D, int NT, Share SHARE, Units UNITS>
__device__ __forceinline__ void run(const AttnArgs &a, unsigned char *sm) {
  constexpr bool MANY = UNITS != kFewUnits;
  using SM = Smem<D, NT, MANY>;
  using S = Shape8<NT, SHARE>;
  constexpr bool SOLO = SHARE != kKeys;  // a warp has whole rows by itself
  constexpr int kSlices = S::kTile / kSlice;
  constexpr int kStride = SOLO ? 1 : kWarps;  // steps from one of a warp's to the next
  constexpr int kSteps = D / 16;          // of 16 elements
  constexpr int kWords = D / 16;          // 32-bit words of a key that a thread takes
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_addr(sm) + warp * SM::kStages * SM::kSliceBytes;
  float *scales = reinterpret_cast<float *>(sm + SM::kScale) + warp * SM::kStages * 2;
  float *factor = reinterpret_cast<float *>(sm + SM::kFactor) + (SOLO ? warp * NT * 8 : 0);
  [[maybe_unused]] float *join = reinterpret_cast<float *>(sm + SM::kJoin);
  const uint32_t q_at = smem_addr(sm + SM::kQ) + (SOLO ? warp * SM::kQBytes : 0);
  // what the plan deals to: blocks, or warps
  const int me = SHARE == kUnits ? blockIdx.x * kWarps + warp : blockIdx.x, all = SHARE == kUnits ? gridDim.x * kWarps : gridDim.x;
  const bool speaks = SHARE == kUnits ? lane == 0 : tid == 0;
  auto meet = [] {
    if constexpr (SOLO) __syncwarp();
    else __syncthreads();
  };
  AttnPlan<S> plan(a.H, SHARE == kHeads ? a.HKV / kWarps : a.HKV, a.plan_coarse, a.plan_least);
  const AttnStaged *staged = reinterpret_cast<const AttnStaged *>(sm);  // until the first copies
  const AttnStart st = attn_start(a, plan, staged, me, all);  // each warp for itself
  AttnWalk<S> walk(a, plan, st, me, all);
  if (a.jobs && speaks) a.jobs[me].rows = 0;
  if (MANY && a.jobs && speaks) a.jobs[me].pad[0] = S::kRows;  // the merge kernel goes by it
  if (UNITS == kForWarps && SHARE != kUnits && a.jobs)  // the merge kernel looks at a job for each warp
    for (int i = all + me * (kWarps - 1) + tid; i < all + (me + 1) * (kWarps - 1); i += kThreads) a.jobs[i].rows = 0;
  __syncthreads();  // what was staged has been read
  const uint64_t once = l2_evict_first();
  // A lane copies a 16-byte piece of every kAtOnce-th row of a step.
  constexpr int kChunks = D / 16, kAtOnce = 32 / kChunks, kCopies = kSlice / kAtOnce;
  const int my_row = lane / kChunks, chunk = lane % kChunks;
  const long long row_bytes = (long long)a.HKV * D, rows_apart = kAtOnce * row_bytes;
  uint32_t copy_to[kCopies];  // within a stage
#pragma unroll
  for (int j = 0; j < kCopies; j++) {
    const int r = j * kAtOnce + my_row;
    copy_to[j] = ring + r * D + ((chunk ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
  }
  const int scale_blocks = a.page_size / kScaleBlock;
  AttnUnit u;
  while (walk.next(u)) {
    if (u.slot >= 0 && !a.jobs) {  // a cut unit has no place: never by the plan
      if (speaks && a.flags) atomicOr(a.flags, kFlagLaunchConfig);
      continue;
    }
    if (speaks && u.slot == 2 * me + 1) {
      AttnJob job = attn_job(u);
      job.pad[0] = S::kRows;
      a.jobs[me] = job;
    }
    if constexpr (SHARE == kHeads) {  // this warp's
      u.gp /= kWarps;
      u.kvh = u.kvh * kWarps + warp;
      u.head0 += warp * u.gp;
    }
    meet();  // the previous unit's (or the plan's) shared memory has been read
    const int end = min(u.t1 * S::kTile, max(u.pos0 + u.n_tok, 0));  // behind the last key that anybody sees
    const int first = u.t0 * kSlices + (SOLO ? 0 : warp), n_slices = (end + kSlice - 1) / kSlice;
    const int steps = n_slices > first ? (n_slices - first + kStride - 1) / kStride : 0;  // this warp's
    // The pages of 32 steps, a lane each.
    int page = 0;
    auto look_up = [&](int i) {
      const int key = (first + min(i + lane, steps - 1) * kStride) * kSlice;
      page = __ldg(a.table + (long long)u.seq * a.max_pages + (a.page_log >= 0 ? key >> a.page_log : key / a.page_size));
      if ((unsigned)page >= (unsigned)a.n_pages) {  // reads as zeros
        page = -1;
        if (a.flags && i + lane < steps) atomicOr(a.flags, kFlagBadSeqlens);
      }
    };
    const long long lane_from = (long long)u.kvh * D + my_row * row_bytes + chunk * 16;
    int to_stage = 0;
    auto fetch = [&](int i) {  // step i, into the next stage; an empty group behind the last one
      if (i < steps) {
        if ((i & 31) == 0) look_up(i);
        const int mine = __shfl_sync(0xffffffffu, page, i & 31), at_page = max(mine, 0);
        const int key = (first + i * kStride) * kSlice;
        const int inside = a.page_log >= 0 ? key & (a.page_size - 1) : key % a.page_size;
        const long long from = ((long long)at_page * a.page_size + inside) * row_bytes + lane_from;
        const char *k = static_cast<const char *>(a.k) + from, *v = static_cast<const char *>(a.v) + from;
        const uint32_t stage = to_stage * SM::kSliceBytes;
        if (mine >= 0 && key + kSlice <= u.len) {
#pragma unroll
          for (int j = 0; j < kCopies; j++) {
            copy16(copy_to[j] + stage, k + j * rows_apart, once);
            copy16(copy_to[j] + stage + kSlice * D, v + j * rows_apart, once);
          }
        } else {
          const int rows = mine < 0 ? 0 : u.len - key;
#pragma unroll
          for (int j = 0; j < kCopies; j++) {
            const bool valid = j * kAtOnce + my_row < rows;
            const long long at = valid ? from + j * rows_apart : 0;
            copy16(copy_to[j] + stage, static_cast<const char *>(a.k) + at, once, valid ? 16 : 0);
            copy16(copy_to[j] + stage + kSlice * D, static_cast<const char *>(a.v) + at, once, valid ? 16 : 0);
          }
        }
        if (lane < 2)
          cp_async4(smem_addr(scales + to_stage * 2 + lane),
                    (lane ? a.v_scale : a.k_scale) + ((long long)at_page * scale_blocks + inside / kScaleBlock) * a.HKV + u.kvh, mine < 0 ? 0 : 4);
        to_stage = to_stage == SM::kStages - 1 ? 0 : to_stage + 1;
      }
      copies_end();
    };
#pragma unroll
    for (int i = 0; i < SM::kStages - 1; i++) fetch(i);
    // Q's fragments: row r of group nt, for k step s the elements 2 D / 8 t' + 4 s .. + 3
    // of thread t' of a row.  A warp has whole rows, so that each row's largest
    // exponent is at hand.
    constexpr int kMine = SOLO ? NT * 8 : NT;  // rows of a warp
    auto row_of = [&](int i) { return SOLO ? i : warp + i * kWarps; };
    uint2 q[kMine];  // 4 elements for each lane (d = 64: lanes 0-15)
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int r = row_of(i), tok = r / u.gp;
      q[i] = make_uint2(0, 0);
      if (tok < u.n_tok && lane * 4 < D)
        q[i] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.q) + (long long)(u.row0 + tok) * a.q_stride +
                                                     (u.head0 + r % u.gp) * D + lane * 4));
    }
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int r = row_of(i);
      const uint2 x = q[i];
      const uint32_t lo0 = x.x << 16, hi0 = x.x & 0xffff0000u, lo1 = x.y << 16, hi1 = x.y & 0xffff0000u;
      const uint32_t top = __reduce_max_sync(0xffffffffu, max(max(lo0 & 0x7fffffffu, hi0 & 0x7fffffffu), max(lo1 & 0x7fffffffu, hi1 & 0x7fffffffu)));
      // 2^up brings the largest element to [2^14, 2^15); non-finite rows stay as they are
      const int e = (int)(top >> 23) - 127, up = e == 128 ? 0 : max(14 - e, -113);
      const float f1 = __int_as_float((127 + up / 2) << 23), f2 = __int_as_float((127 + up - up / 2) << 23);
      auto scaled = [&](uint32_t y) { return __uint_as_float(y) * f1 * f2; };
      if (lane * 4 < D) {
        // thread t' has elements t' D / 4 ..: 4 of them a k step
        const int owner = lane / (D / 16), step = lane % (D / 16);
        const uint32_t to = q_at + (((r >> 3) * kSteps + (step & ~1)) * 32 + 2 * ((r & 7) * 4 + owner) + (step & 1)) * 8;
        const uint32_t b0 = pack_f16(scaled(lo0), scaled(hi0)), b1 = pack_f16(scaled(lo1), scaled(hi1));
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(b0), "r"(b1) : "memory");
      }
      // scale log2(e) 2^-up: of the scores
      if (lane == 0) factor[r] = a.scale_log2 * __int_as_float((127 - up / 2) << 23) * __int_as_float((127 - up + up / 2) << 23);
    }
    meet();
    float o[NT][D / 16][4];
    // Of a row: the maximum of the scores and that of them with V's scale (powers of
    // two), the sum of the weights, the factor of V's scale in weights, of K's in scores.
    float m[NT][2], mv[NT][2], l[NT][2], ratio[NT][2], f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
      for (int i = 0; i < D / 16; i++)
#pragma unroll
        for (int c = 0; c < 4; c++) o[n][i][c] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; c++) {
        const int r = n * 8 + 2 * t + c;
        m[n][c] = mv[n][c] = kNone;
        l[n][c] = ratio[n][c] = 0.f;
        f[n][c] = factor[r];
      }
    }
    int stage = 0;
    for (int i = 0; i < steps; i++) {
      copies_wait<SM::kStages - 2>();
      __syncwarp();  // step i is there, and step i - 1 has been read
      fetch(i + SM::kStages - 1);
      const uint32_t at = ring + stage * SM::kSliceBytes;
      const float2 scale = *reinterpret_cast<const float2 *>(scales + stage * 2);
      stage = stage == SM::kStages - 1 ? 0 : stage + 1;
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      {
        uint32_t k0[kWords], k1[kWords];  // keys g and g + 8
#pragma unroll
        for (int w = 0; w < kWords; w += 4) {
          const int c = D == 128 ? (2 * t + w / 4) ^ g : t ^ ((g >> 1) & 3);
          const uint4 x = lds128(at + g * D + c * 16), y = lds128(at + (g + 8) * D + c * 16);
          k0[w] = x.x; k0[w + 1] = x.y; k0[w + 2] = x.z; k0[w + 3] = x.w;
          k1[w] = y.x; k1[w + 1] = y.y; k1[w + 2] = y.z; k1[w + 3] = y.w;
        }
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint4 b[NT];  // two steps' of Q
#pragma unroll
          for (int n = 0; n < NT; n++) b[n] = lds128(q_at + ((n * kSteps + k) * 32 + 2 * lane) * 8);
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const uint32_t a0 = half_lo(k0[k + e]), a1 = half_lo(k1[k + e]), a2 = half_hi(k0[k + e]), a3 = half_hi(k1[k + e]);
#pragma unroll
            for (int n = 0; n < NT; n++) mma(s[n], a0, a1, a2, a3, e ? b[n].z : b[n].x, e ? b[n].w : b[n].y);
          }
        }
      }
      // s[n][0], [1]: key g of rows 2 t, 2 t + 1; [2], [3]: key g + 8
      const int key = (first + i * kStride) * kSlice;
      if (key + kSlice - 1 > u.pos0) {  // some row does not see all of them
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int c = 0; c < 2; c++) {
            const int limit = u.pos0 + min((n * 8 + 2 * t + c) / u.gp, u.n_tok - 1);
            if (key + g > limit) s[n][c] = -CUDART_INF_F;
            if (key + g + 8 > limit) s[n][2 + c] = -CUDART_INF_F;
          }
      }
      // V's scale is below 2^(fv + 1); not below -117, so that `ratio` is finite for a zero one too
      const float fv = (float)max((int)(__float_as_uint(scale.y) >> 23 & 255) - 127, -117);
      bool move = false;
      float fk[NT][2];
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
          fk[n][c] = fmaxf(f[n][c] * scale.x, 1e-37f);  // -inf times it stays that
          const float top = fmaxf(s[n][c], s[n][2 + c]) * fk[n][c] - kLag;
          move |= top > m[n][c] || top + fv > mv[n][c];
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int c = 0; c < 2; c++) {
            float top = fmaxf(s[n][c], s[n][2 + c]) * fk[n][c];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m[n][c], top), vn = fmaxf(mv[n][c], top + fv);
            const bool some = mn > kNone;  // something is visible by now
            l[n][c] *= some ? ex2(m[n][c] - mn) : 0.f;
            const float down = some ? ex2(mv[n][c] - vn) : 0.f;
            ratio[n][c] = some ? ex2(mn - vn + kShift) : 0.f;
            m[n][c] = mn;
            mv[n][c] = vn;
#pragma unroll
            for (int j = 0; j < D / 16; j++) {
              o[n][j][c] *= down;
              o[n][j][2 + c] *= down;
            }
          }
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int n = 0; n < NT; n++) {
        float w[4];
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const float p0 = ex2(fmaf(s[n][c], fk[n][c], -m[n][c])), p1 = ex2(fmaf(s[n][2 + c], fk[n][c], -m[n][c]));
          // finite: where a row has met zero values alone so far (`ratio` up to 2^123) and large
          // ones come that it does not see, 0 times this is 0
          const float fw = fminf(scale.y * ratio[n][c], 0x1p126f);
          l[n][c] += p0 + p1;
          w[c] = p0 * fw;
          w[2 + c] = p1 * fw;
        }
        p[n][0] = transpose8(pack_f16(w[0], w[1]));
        p[n][1] = transpose8(pack_f16(w[2], w[3]));
      }
      // V^T: elements g D / 8 .. of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9; products 2 j and
      // 2 j + 1 of 16 x 8 take the elements 4 j .. + 3
      constexpr int kWordsV = D / 32;
      uint32_t v[4][kWordsV];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int r = 2 * t + (j & 1) + (j >> 1) * 8;
        if constexpr (D == 128) {
          const uint4 x = lds128(at + kSlice * D + r * D + ((g ^ (r & 7)) << 4));
          v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
        } else {
          const uint2 x = lds64(at + kSlice * D + r * D + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
          v[j][0] = x.x; v[j][1] = x.y;
        }
      }
#pragma unroll
      for (int w = 0; w < kWordsV; w++) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t x = __byte_perm(v[0][w], v[1][w], h ? 0x7362 : 0x5140), y = __byte_perm(v[2][w], v[3][w], h ? 0x7362 : 0x5140);
          const uint32_t a0 = half_lo(x), a1 = half_hi(x), a2 = half_lo(y), a3 = half_hi(y);
#pragma unroll
          for (int n = 0; n < NT; n++) mma(o[n][2 * w + h], a0, a1, a2, a3, p[n][0], p[n][1]);
        }
      }
    }
    copies_wait<0>();
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int c = 0; c < 2; c++)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);
    const int rows = u.n_tok * u.gp;
    const bool part = u.slot >= 0;
    bool finite = true;
    if constexpr (SOLO) {
      // a thread has D / 8 elements in a row of two rows of each group
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const int r = n * 8 + 2 * t + c;
          if (r >= rows) continue;
          const float top = m[n][c] <= kNone ? -CUDART_INF_F : m[n][c], sum = l[n][c];
          const float back = ex2(mv[n][c] - m[n][c] - kShift), by = part ? back : sum == 0.f ? 0.f : back / sum;
          float y[D / 8];
#pragma unroll
          for (int j = 0; j < D / 16; j++) {
            y[2 * j] = o[n][j][c] * by;
            y[2 * j + 1] = o[n][j][2 + c] * by;
          }
          const long long at = (long long)(u.row0 + r / u.gp) * a.H + u.head0 + r % u.gp;
          if (part) {
            const long long to = (long long)u.slot * S::kRows + (SHARE == kHeads ? (r / u.gp * kWarps + warp) * u.gp + r % u.gp : r);
#pragma unroll
            for (int j = 0; j < D / 8; j += 4)
              a.part_o[to * (D / 4) + g * (D / 32) + j / 4] = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
            if (g == 0) a.part_ml[to] = make_float2(top, sum);
          } else {
            uint32_t z[D / 16];
#pragma unroll
            for (int j = 0; j < D / 16; j++) {
              finite &= fabsf(y[2 * j]) < kBf16Inf && fabsf(y[2 * j + 1]) < kBf16Inf;
              const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
              z[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
            uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + g * (D / 8));
#pragma unroll
            for (int j = 0; j < D / 16; j += 4) to[j / 4] = make_uint4(z[j], z[j + 1], z[j + 2], z[j + 3]);
            if (g == 0 && a.lse) a.lse[at] = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.69314718056f;
          }
        }
      if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
      continue;
    }
    // ---- the eight warps' results, joined in order
    __syncthreads();  // every warp's ring has been read
    float *place = reinterpret_cast<float *>(sm) + warp * NT * 8 * SM::kRow;
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int c = 0; c < 2; c++) {
        const int r = n * 8 + 2 * t + c;
        if (r >= rows) continue;
        float *to = place + r * SM::kRow + g * (D / 8);
#pragma unroll
        for (int j = 0; j < D / 16; j += 2)
          *reinterpret_cast<float4 *>(to + 2 * j) = make_float4(o[n][j][c], o[n][j][2 + c], o[n][j + 1][c], o[n][j + 1][2 + c]);
        if (g == 0) {
          float *x = join + (warp * NT * 8 + r) * 3;
          x[0] = m[n][c];
          x[1] = l[n][c];
          x[2] = mv[n][c];
        }
      }
    __syncthreads();
    for (int item = tid; item < rows * (D / 4); item += kThreads) {
      const int r = item / (D / 4), d4 = item % (D / 4);
      float top = kNone, top_v = kNone, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        top = fmaxf(top, join[(w * NT * 8 + r) * 3]);
        top_v = fmaxf(top_v, join[(w * NT * 8 + r) * 3 + 2]);
      }
      const float base = top;
      // of the smallest values a factor could vanish: 2^64 too large then, and made good at the end
      const bool tiny = top_v - base < -64.f;
      const float shift = tiny ? kShift - 64.f : kShift;
      if (top <= kNone) top = -CUDART_INF_F;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        const float *x = join + (w * NT * 8 + r) * 3;
        sum += x[1] * ex2(x[0] - base);
        const float fo = ex2(x[2] - base - shift);
        const float4 z = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sm) + (w * NT * 8 + r) * SM::kRow + d4 * 4);
        y.x += fo * z.x; y.y += fo * z.y; y.z += fo * z.z; y.w += fo * z.w;
      }
      if (tiny) {
        y.x *= 0x1p-64f; y.y *= 0x1p-64f; y.z *= 0x1p-64f; y.w *= 0x1p-64f;
      }
      if (part) {
        a.part_o[MANY ? ((long long)u.slot * S::kRows + r) * (D / 4) + d4 : ((long long)u.slot * (D / 4) + d4) * S::kRows + r] = y;
        if (d4 == 0) a.part_ml[(long long)u.slot * S::kRows + r] = make_float2(top, sum);
      } else {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        y.x *= inv; y.y *= inv; y.z *= inv; y.w *= inv;
        finite &= fabsf(y.x) < kBf16Inf && fabsf(y.y) < kBf16Inf && fabsf(y.z) < kBf16Inf && fabsf(y.w) < kBf16Inf;
        const long long at = (long long)(u.row0 + r / u.gp) * a.H + u.head0 + r % u.gp;
        __nv_bfloat162 z[2] = {__floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + d4 * 4) = *reinterpret_cast<uint2 *>(z);
        if (d4 == 0 && a.lse) a.lse[at] = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.69314718056f;
      }
    }
    if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
  }
}

// With units enough a block has eight heads of a sequence at a time, a warp each: its
// warps read neighbouring 128-byte rows at about the same time, which memory gives faster
// than rows 1 KB apart, and nothing is joined but what the plan has cut.  256 sequences of
// up to 4096 keys, 32/8 heads of 128, 215 us as blocks of one head's, 186 so; 64 over 4096
// keys 105 and 90; 128 over 4096, 32/32 heads, 751 and 632.  (The heads of all sequences one
// after the other instead, so that blocks read neighbouring rows, gave 212 for 215.)
// With units for thousands of warps, short ones are a warp's each: 256 sequences over 300
// keys, 8 key/value heads, 54.7 us as blocks', 34.5 as warps'; 1000 over 50 keys 104 and 57;
// but 256 over 1000, 16 heads, 192 and 205, since 2432 warps each somewhere else in its unit
// read memory in a worse order.
constexpr int kShort = 6;      // key tiles of a unit, on average
constexpr int kShortTeam = 1;  // where eight heads may be a unit (2000 over 300: 266 us, 231 as teams')
template <int D, int NT, Units UNITS>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<NT>()) gdn_attn8_kernel(const AttnArgs a) {
  extern __shared__ __align__(128) unsigned char sm[];
  AttnStaged *staged = reinterpret_cast<AttnStaged *>(sm);
  attn_stage<kThreads, Shape8<NT>>(a, staged, blockIdx.x);
  asm volatile("griddepcontrol.launch_dependents;");  // the merge kernel waits for this one's end
  __syncthreads();
  if constexpr (UNITS != kFewUnits) {
    // every warp for itself, of the first kStaged sequences
    uint32_t tiles = 0, seqs = 0;
    for (int n = threadIdx.x & 31; n < a.n_seqs && n < kStaged; n += 32)
      if (staged[n].nq > 0) {
        tiles += (uint32_t)AttnPlan<SoloShape8>::tiles(staged[n].base + staged[n].nq);
        seqs++;
      }
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    seqs = __reduce_add_sync(0xffffffffu, seqs);
    // (without places for partial results there is a warp or block for each unit)
    if (UNITS == kForWarps && (!a.jobs || tiles <= (a.HKV % kWarps == 0 ? kShortTeam : kShort) * (unsigned long long)seqs)) run<D, NT, kUnits, kForWarps>(a, sm);
    else if (a.HKV % kWarps == 0 && a.jobs) run<D, NT, kHeads, UNITS>(a, sm);
    else run<D, NT, kKeys, UNITS>(a, sm);
  } else {
    run<D, NT, kKeys, kFewUnits>(a, sm);
  }
  // Behind the kernel for many rows this one begins as that one's blocks end (2 chunks of
  // up to 500 tokens among 14 single ones 154 -> 150 us): what follows waits for both.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the pieces of a unit that a block or warp of the plan began and did not end, in
// their order: a thread has four columns of a row.  There are `jobs` of them; eight blocks
// share one where a unit is eight heads', of which there are `teams` (64 sequences over 4096
// keys of 8 heads, five pieces each: 98 us in all with a block for each, 90 so).
constexpr int kMergeThreads = 128;
static_assert(TeamShape8::kRows <= kWarps * SoloShape8::kRows, "places for warps' units are enough for teams'");
template <int D>
__global__ void __launch_bounds__(kMergeThreads) gdn_attn8_merge_kernel(const AttnArgs a, const int jobs, const int teams) {
  // launched while the attention kernel runs; its results are there after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int part = blockIdx.x / teams, of_team = blockIdx.x - part * teams;
  const bool shared = a.jobs[of_team].pad[0] == TeamShape8::kRows;
  const int first = shared ? of_team : blockIdx.x;  // block or warp of the plan
  if (first >= jobs) return;
  const AttnJob job = a.jobs[first];
  const int row0 = shared ? (job.rows + 7) / 8 * part : 0, rows = shared ? min(job.rows, (job.rows + 7) / 8 * (part + 1)) : job.rows;
  const int n = job.last - first + 1;  // pieces
  auto slot = [&](int i) { return (long long)(i == 0 ? 2 * first + 1 : 2 * (first + i)); };
  bool finite = true;
  for (int item = row0 * (D / 4) + threadIdx.x; item < rows * (D / 4); item += kMergeThreads) {
    const int r = item / (D / 4), d4 = item % (D / 4);
    float top = -CUDART_INF_F, sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += 4) {
      float2 ml[4];
      float4 x[4];
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const long long at = slot(i0 + k < n ? i0 + k : i0) * job.pad[0] + r;
        ml[k] = i0 + k < n ? a.part_ml[at] : make_float2(-CUDART_INF_F, 0.f);
        x[k] = a.part_o[at * (D / 4) + d4];
      }
      float next = top;
#pragma unroll
      for (int k = 0; k < 4; k++) next = fmaxf(next, ml[k].x);
      const float base = next == -CUDART_INF_F ? 0.f : next, down = ex2(top - base);
      sum *= down;
      y.x *= down; y.y *= down; y.z *= down; y.w *= down;
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (i0 + k < n) {
          const float f = ex2(ml[k].x - base);
          sum += f * ml[k].y;
          y.x += f * x[k].x; y.y += f * x[k].y; y.z += f * x[k].z; y.w += f * x[k].w;
        }
      top = next;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    y.x *= inv; y.y *= inv; y.z *= inv; y.w *= inv;
    finite &= fabsf(y.x) < kBf16Inf && fabsf(y.y) < kBf16Inf && fabsf(y.z) < kBf16Inf && fabsf(y.w) < kBf16Inf;
    const long long at = (long long)(job.row0 + r / job.gp) * a.H + job.head0 + r % job.gp;
    __nv_bfloat162 z[2] = {__floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + d4 * 4) = *reinterpret_cast<uint2 *>(z);
    if (d4 == 0 && a.lse) a.lse[at] = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.69314718056f;
  }
  if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
}

template <int D, int NT, Units UNITS>
std::atomic<uint64_t> allowed{0};

// behind: the kernel for many rows has just been launched, on other sequences
template <int D, int NT, Units UNITS>
cudaError_t launch(const AttnArgs &a, const AttnLaunch &l, bool behind, cudaStream_t stream) {
  constexpr int kBytes = Smem<D, NT, UNITS != kFewUnits>::kBytes;
  const cudaError_t e = allow_smem(reinterpret_cast<const void *>(&gdn_attn8_kernel<D, NT, UNITS>), kBytes, allowed<D, NT, UNITS>);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(UNITS == kForWarps ? (l.blocks + kWarps - 1) / kWarps : l.blocks);
  config.blockDim = dim3(kThreads);
  config.dynamicSmemBytes = kBytes;
  config.stream = stream;
  config.attrs = &early;
  config.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&config, gdn_attn8_kernel<D, NT, UNITS>, a);
}

template <int D>
cudaError_t launch_few(const Attn8Launch &l, cudaStream_t stream) {
  const AttnLaunch &f = l.few_launch;
  if (l.groups == 4) return launch<D, 4, kFewUnits>(l.few, f, l.has_many, stream);
  if (l.groups == 2) return launch<D, 2, kFewUnits>(l.few, f, l.has_many, stream);
  if (l.warps) return launch<D, 1, kForWarps>(l.few, f, l.has_many, stream);
  return l.teams ? launch<D, 1, kForBlocks>(l.few, f, l.has_many, stream) : launch<D, 1, kFewUnits>(l.few, f, l.has_many, stream);
}

// Joins what a plan has cut.
// by_rows: partial results lie row by row; warps: the plan deals to warps
cudaError_t join(const AttnArgs &a, int d, const AttnLaunch &l, bool by_rows, bool warps, cudaStream_t stream) {
  if (!l.split || l.blocks < 2) return cudaSuccess;
  if (!by_rows) return launch_attn8_merge(a, d, l.rows, l.blocks, stream);
  // may be set up while the attention kernel still runs
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  const int teams = warps ? l.blocks / kWarps : l.blocks;
  config.gridDim = dim3(kWarps * teams - 1);
  config.blockDim = dim3(kMergeThreads);
  config.stream = stream;
  config.attrs = &early;
  config.numAttrs = 1;
  return d == 64 ? cudaLaunchKernelEx(&config, gdn_attn8_merge_kernel<64>, a, l.blocks, teams)
                 : cudaLaunchKernelEx(&config, gdn_attn8_merge_kernel<128>, a, l.blocks, teams);
}

}  // namespace

bool attn8_launch(const AttnArgs &a, int d, Attn8Launch &l) {
  const long long G = a.H / a.HKV, most = (a.cu ? (long long)a.Ttot : (long long)a.T) * G;  // rows of a sequence
  // Up to 32 rows: 64 sequences over 4096 keys, 8 key/value heads of 128, with 20 to 32
  // rows each take 250 us as many ones, 170 to 177 as few.  In a packed call most sequences
  // have one token, G rows, which the kernel for 16 does faster.
  // A call of little work, as far as the host knows, is left to the kernel for few rows
  // altogether, which has longer sequences 16 rows at a time: one kernel's launches, and a
  // start without tensor maps and tensor memory.  One chunk of 64 tokens over 4000 keys, 32/8
  // heads (8.2e6 rows times keys times heads) 36.5 us so, 43.7 as many rows; 16 over 30000
  // (15e6) 53 and 55; 32 over 16000 (16e6) 56 and 45.
  const bool small = (double)a.Ttot * G * a.max_len * a.HKV <= 1e7;
  const int limit = small ? INT32_MAX : a.cu && G <= 16 ? 16 : 32;
  l.few = l.many = a;
  l.few.few_rows = l.many.few_rows = limit;
  l.has_few = a.cu ? G <= limit : most <= limit;
  l.has_many = most > limit;
  l.groups = a.cu ? (G <= 16 ? 2 : 4) : most <= 8 ? 1 : most <= 16 || most > 32 ? 2 : 4;
  l.few_launch = l.many_launch = AttnLaunch{};
  // Enough units that a warp's equal share is not a small part of one: its pieces are few.
  // Where eight heads may be a unit, nearly one for each warp (of 2432): 100 sequences over
  // 1000 keys, 16 key/value heads, 82 us as warps', 71 as teams'; 256 over 300, 8 heads, 34.5
  // and 39.7.  With fewer than 48 units of eight heads each is in many pieces: 32 sequences
  // over 4000 keys 47 us as blocks', 50 as teams'; 48 of them 80 and 71.
  const int blocks = blocks_per_sm<2>() * sm_count();
  l.warps = l.groups == 1 && (a.HKV % kWarps == 0 ? 1.25 : 4.) * a.n_seqs * a.HKV >= (double)blocks * kWarps;
  l.teams = l.groups == 1 && !l.warps && a.HKV % kWarps == 0 && (long long)a.n_seqs * (a.HKV / kWarps) >= 48;
  if (l.has_few)
    l.few_launch = l.warps ? attn_plan_launch<SoloShape8>(l.few, blocks * kWarps)
                   : l.teams ? attn_plan_launch<TeamShape8>(l.few, blocks)
                   : l.groups == 4 ? attn_plan_launch<Shape8<4>>(l.few, blocks_per_sm<4>() * sm_count())
                                   : attn_plan_launch<Shape8<2>>(l.few, blocks);
  if (l.has_many) l.many_launch = attn_plan_launch<TcShape8>(l.many, sm_count());
  return (!l.has_few || l.few_launch.blocks > 0) && (!l.has_many || l.many_launch.blocks > 0);
}

cudaError_t launch_attn8(const Attn8Launch &l, int d, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (l.has_many) e = launch_attn8_tc(l.many, d, l.many_launch.blocks, stream);
  if (e == cudaSuccess && l.has_few) e = d == 64 ? launch_few<64>(l, stream) : launch_few<128>(l, stream);
  if (e == cudaSuccess && l.has_many) e = join(l.many, d, l.many_launch, false, false, stream);
  if (e == cudaSuccess && l.has_few) e = join(l.few, d, l.few_launch, l.warps || l.teams, l.warps, stream);
  return e;
}

}  // namespace gdn
