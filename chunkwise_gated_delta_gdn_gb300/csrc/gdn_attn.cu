// gdn_attn.cu -- causal softmax attention with grouped heads, over a whole
// prompt or over a paged cache: the fp32 kernel, the merge of partial results
// (both types) and the launch (bf16: gdn_attn_tc.cu).
//
//   s_j = scale q.k_j (j <= p), m = max_j s_j, l = sum_j e^(s_j - m),
//   o = sum_j e^(s_j - m) v_j / l,  lse = m + ln l
//
// One pass over the keys with the running maximum and sum; what a row has when
// no key is visible to it (o = 0, lse = -inf) follows from l = 0.
#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "gdn_attn.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace {

// fp32: a unit of 64 rows, 64 keys per step, four warps of 16 rows, both
// products in fp32 multiply-adds: 125 us for 2 x 1023 tokens, 16 heads of 64; 1095
// for ten prompts of 2199 tokens, 4 heads of 128 (35 and 45 TFLOP/s of 74).
// Products of split operands on the tensor cores (three tf32 ones each, on
// mma.sync) took 159 us for the first, with several times the error, since those
// accumulations are cut off and not rounded.  The error against 64 bits is that
// of plain 32-bit operations, 6e-7 at 1023 tokens and 1.2e-6 at 8192; sums of 16
// products and of a tile's keys by themselves would make it 4e-7 (126 and 1106 us;
// 200-token prompts a tenth slower).
//
// S = Q K^T: a thread has 8 rows, as pairs, and 4 keys 16 apart; queries lie
// transposed in shared memory, keys as they come.  The 16 threads of a row are
// half a warp.  O = P V: the weights go through shared memory, and a thread has 8
// rows and D / 16 columns.  The next keys are on their way while a tile's weights
// are made and used, the next values during its scores.  What is left: 57% of the
// multiply-adds' clocks are used, and the instructions around them (reads of
// shared memory, the second copy of a pair's factor) wait for one another; more
// warps do not fit the registers.  One multiply-add to an instruction: 135 us where
// pairs took 134, 1243 where they took 1151.  Loops unrolled 2 and 8 fold: 131 and
// 1095; 4 and 16: these figures; 8 and 32: 127 and 1100.
//
// At most 16 rows (a decode step): every warp has them, and 16 of the 64 keys.  32
// sequences over 8192 keys, 8 heads of 128: 572 us, 3.8 TB/s; one over 300, 16 us.
// A tile of theirs takes as long as one of 64 rows (both wait for loads): with
// 1/2 and 1/3 of its cost, chunks among single tokens took 1.5 times as long.  A
// unit's start and end take half a tile (with a quarter, ten prompts of 2199
// tokens 1129 us).  Units of up to two tiles stay whole where each gets a block: a
// 100-token prompt takes 18 us with its launch, cut and joined 28; one of 200, 39
// whole and 27 cut.
using WarpShape = AttnShape<64, 64, 64, 2, 1, 2, 1, 16, 0, 1>;
constexpr int kThreads = 128;

template <int D>
struct WarpSmem {
  static constexpr int kKRow = D + 4;         // floats from one key to the next: 8 lanes hit 32 banks
  static constexpr int kQ = 0;                // [D][64], queries transposed
  static constexpr int kK = 64 * D;           // [64][kKRow]
  static constexpr int kV = kK + 64 * kKRow;  // [64][D]
  static constexpr int kP = kV + 64 * D;      // [warp][64 keys][16 rows]
  static constexpr int kBytes = (kP + 4 * 64 * 16) * 4;
};
static_assert(kStaged * sizeof(AttnStaged) + kThreads * sizeof(AttnChunk) <= WarpSmem<64>::kBytes, "staging");
template <int D>
constexpr int blocks_per_sm() { return D == 64 ? 3 : 2; }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void get4(float *x, const float *p) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

// eight values as four pairs
__device__ __forceinline__ void get_pairs(uint64_t *x, const float *p, const float *p4) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p), b = *reinterpret_cast<const ulonglong2 *>(p4);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
// 16 bytes from global to shared memory, in the background; zeros when !valid
__device__ __forceinline__ void copy16(float *to, const float *from, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until all groups but the last N are there
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<D>()) gdn_attn_warp_kernel(const AttnArgs a) {
  using SM = WarpSmem<D>;
  constexpr int kCols = D / 16;  // columns of a thread: 4 from 4 cg on, and for D = 128 4 from 64 + 4 cg on
  extern __shared__ __align__(16) float smem[];
  float *Qt = smem + SM::kQ, *Ks = smem + SM::kK, *Vs = smem + SM::kV;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rg = lane >> 4, cg = lane & 15;  // rows rg * 8 .. + 7 of the warp's 16; keys cg, cg + 16, ..
  float *P = smem + SM::kP + warp * 64 * 16;
  // weights of key j, rows 4 c .. 4 c + 3: the four chunks of a key are swapped
  // about so that 8 keys' lie in different banks
  auto chunk = [&](int j, int c) { return P + j * 16 + ((c ^ (j >> 1)) & 3) * 4; };
  AttnPlan<WarpShape> plan(a.H, a.HKV, a.plan_coarse, a.plan_least);
  AttnStaged *staged = reinterpret_cast<AttnStaged *>(smem);  // until the first operands
  attn_stage<kThreads>(a, staged, blockIdx.x);
  __syncthreads();
  const AttnStart st = attn_start(a, plan, staged, blockIdx.x, gridDim.x);  // each warp for itself
  AttnWalk<WarpShape> walk(a, plan, st, blockIdx.x, gridDim.x);
  AttnUnit u;
  if (a.jobs && tid == 0) a.jobs[blockIdx.x].rows = 0;
  while (walk.next(u)) {
    if (u.slot >= 0 && !a.jobs) {  // a cut unit has no place: never by the plan
      if (tid == 0 && a.flags) atomicOr(a.flags, kFlagLaunchConfig);
      continue;
    }
    if (tid == 0 && u.slot == 2 * (int)blockIdx.x + 1) a.jobs[blockIdx.x] = attn_job(u);
    __syncthreads();  // the previous unit's operands (or the plan's) are read
    const int end = min(u.t1 * 64, max(u.pos0 + u.n_tok, 0));  // behind the last key that anybody sees
    // where a key's row begins; a bad page reads as zeros (-1)
    auto row_of = [&](int key, long long stride) -> long long {
      if (key >= u.len) return -1;
      // a prompt's keys are its own tokens
      if (!a.table) return (u.row0 - u.pos0 + key) * stride + u.kvh * D;
      const int index = a.page_log >= 0 ? key >> a.page_log : key / a.page_size;
      const int page = __ldg(a.table + (long long)u.seq * a.max_pages + index);
      if (page < 0 || page >= a.n_pages) {
        if (a.flags) atomicOr(a.flags, kFlagBadSeqlens);
        return -1;
      }
      return (((long long)page * a.page_size + key - index * a.page_size) * a.HKV + u.kvh) * D;
    };
    // 64 rows from key0 on into shared memory, on their way while others are
    // worked on; one group of copies, empty behind the last tile.  Each lane looks
    // up two rows, all at once, for the whole warp: looked up for each copy, the
    // page numbers' latency was most of a decode step.
    auto fetch = [&](int key0, const void *base, long long stride, float *to, int row_floats) {
      if (key0 < end) {
        constexpr int kRow = D / 4, kStep = kThreads / kRow;  // 16-byte pieces of a row, rows at a time
        const long long low = row_of(key0 + lane, stride), high = row_of(key0 + 32 + lane, stride);
#pragma unroll
        for (int r0 = 0; r0 < 64; r0 += kStep) {
          const int r = r0 + tid / kRow, c = tid % kRow * 4;
          const long long at = __shfl_sync(0xffffffffu, r0 < 32 ? low : high, r & 31);
          copy16(to + r * row_floats + c, static_cast<const float *>(base) + (at < 0 ? 0 : at + c), at >= 0);
        }
      }
      copies_end();
    };
    fetch(u.t0 * 64, a.k, a.k_stride, Ks, SM::kKRow);
    fetch(u.t0 * 64, a.v, a.v_stride, Vs, D);
    {
      const int r = tid & 63, t = r / u.gp;
      const float *q = static_cast<const float *>(a.q) + (long long)(u.row0 + t) * a.q_stride +
                       (u.head0 + r % u.gp) * D;
      for (int c = (tid >> 6) * 4; c < D; c += 8) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < u.n_tok) x = __ldg(reinterpret_cast<const float4 *>(q + c));
        Qt[c * 64 + r] = x.x; Qt[(c + 1) * 64 + r] = x.y;
        Qt[(c + 2) * 64 + r] = x.z; Qt[(c + 3) * 64 + r] = x.w;
      }
    }
    // Few rows: every warp has the same 16 and a quarter of a tile's keys (key cg
    // of its 16 is a thread's), joined at the end.
    const bool few = u.n_tok * u.gp <= 16;
    const int warp_row = few ? 0 : warp * 16;
    uint64_t o[4][kCols] = {};  // pairs of rows
    float m[8], l[8] = {};      // l: this thread's keys only
    int limit[8];               // last visible key
#pragma unroll
    for (int i = 0; i < 8; i++) {
      m[i] = -CUDART_INF_F;
      limit[i] = min(u.pos0 + (warp_row + rg * 8 + i) / u.gp, u.len - 1);
    }
    for (int key0 = u.t0 * 64; key0 < end; key0 += 64) {
      copies_wait<1>();  // the keys
      __syncthreads();
      auto work = [&](auto keys) {
        constexpr int KEYS = decltype(keys)::value;
        float s[8][KEYS];
        {
          uint64_t acc[4][KEYS] = {};  // pairs of rows
          const float *q = Qt + warp_row + rg * 8, *k = Ks + (KEYS == 4 ? cg : warp * 16 + cg) * SM::kKRow;
#pragma unroll 4
          for (int c0 = 0; c0 < D; c0 += 4) {
            float y[KEYS][4];
#pragma unroll
            for (int j = 0; j < KEYS; j++) get4(y[j], k + j * 16 * SM::kKRow + c0);
#pragma unroll
            for (int c = 0; c < 4; c++) {
              uint64_t x[4];
              get_pairs(x, q + (c0 + c) * 64, q + (c0 + c) * 64 + 4);
#pragma unroll
              for (int j = 0; j < KEYS; j++)
#pragma unroll
                for (int i = 0; i < 4; i++) acc[i][j] = fma2(x[i], pair(y[j][c], y[j][c]), acc[i][j]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < KEYS; j++) unpair(acc[i][j], s[2 * i][j], s[2 * i + 1][j]);
        }
        __syncthreads();  // every warp has read the keys
        fetch(key0 + 64, a.k, a.k_stride, Ks, SM::kKRow);
        // running maximum and sum
        const int first = key0 + (KEYS == 4 ? cg : warp * 16 + cg);  // this thread's first key
        float alpha[8];
        const bool all_seen = key0 + 63 <= min(u.pos0, u.len - 1);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          if (!all_seen)
#pragma unroll
            for (int j = 0; j < KEYS; j++)
              if (first + j * 16 > limit[i]) s[i][j] = -CUDART_INF_F;
          float top = s[i][0];
#pragma unroll
          for (int j = 1; j < KEYS; j++) top = fmaxf(top, s[i][j]);
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          top = fmaxf(top, m[i]);
          // Nothing visible yet: weights 0.  The factor between two maxima is that of
          // their rounded products, which the weights were made with: from the
          // unrounded one, errors of 1e-6 in the factor added up with every new
          // maximum (8192 tokens 2.5e-6 of the result, so 1.2e-6).
          const float off = top == -CUDART_INF_F ? 0.f : __fmul_rn(top, a.scale_log2);
          alpha[i] = exp2_approx(__fmul_rn(m[i], a.scale_log2) - off);
          m[i] = top;
          l[i] *= alpha[i];
#pragma unroll
          for (int j = 0; j < KEYS; j++) {
            s[i][j] = exp2_approx(fmaf(s[i][j], a.scale_log2, -off));
            l[i] += s[i][j];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int j = 0; j < kCols; j++) o[i][j] = mul2(o[i][j], pair(alpha[2 * i], alpha[2 * i + 1]));
#pragma unroll
        for (int j = 0; j < KEYS; j++) {
          *reinterpret_cast<float4 *>(chunk(j * 16 + cg, rg * 2)) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
          *reinterpret_cast<float4 *>(chunk(j * 16 + cg, rg * 2 + 1)) = make_float4(s[4][j], s[5][j], s[6][j], s[7][j]);
        }
        copies_wait<1>();  // the values
        __syncthreads();
#pragma unroll 16
        for (int j0 = 0; j0 < 16 * KEYS; j0++) {
          uint64_t x[4];
          float y[kCols];
          get_pairs(x, chunk(j0, rg * 2), chunk(j0, rg * 2 + 1));
          const float *v = Vs + (KEYS == 4 ? j0 : warp * 16 + j0) * D + cg * 4;
          get4(y, v);
          if constexpr (kCols == 8) get4(y + 4, v + 64);
#pragma unroll
          for (int j = 0; j < kCols; j++)
#pragma unroll
            for (int i = 0; i < 4; i++) o[i][j] = fma2(x[i], pair(y[j], y[j]), o[i][j]);
        }
        __syncthreads();  // every warp has read the values
        fetch(key0 + 64, a.v, a.v_stride, Vs, D);
      };
      if (few) work(std::integral_constant<int, 1>{});
      else work(std::integral_constant<int, 4>{});
    }
    float out[8][kCols];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < kCols; j++) unpair(o[i][j], out[2 * i][j], out[2 * i + 1][j]);
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
    if (few) {
      // Warps 1-3 leave their outputs, maxima and sums in the places of the keys
      // and values (no copy is on its way there), warp 0 adds them up in order.
      constexpr int kRow = D + 4, kNext = 16 * kRow;
      float *place = smem + SM::kK + (warp * 16 + rg * 8) * kRow;
      __syncthreads();
      if (warp > 0) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          float *p = place + i * kRow;
#pragma unroll
          for (int b = 0; b < kCols; b += 4)
            *reinterpret_cast<float4 *>(p + cg * 4 + b * 16) =
                make_float4(out[i][b], out[i][b + 1], out[i][b + 2], out[i][b + 3]);
          if (cg == 0) *reinterpret_cast<float2 *>(p + D) = make_float2(m[i], l[i]);
        }
      }
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float *p = place + i * kRow;
          float2 ml[4];
          ml[0] = make_float2(m[i], l[i]);
#pragma unroll
          for (int w = 1; w < 4; w++) ml[w] = *reinterpret_cast<const float2 *>(p + w * kNext + D);
          m[i] = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
          const float off = m[i] == -CUDART_INF_F ? 0.f : __fmul_rn(m[i], a.scale_log2);
          l[i] = 0.f;
#pragma unroll
          for (int w = 0; w < 4; w++) {
            const float f = exp2_approx(__fmul_rn(ml[w].x, a.scale_log2) - off);
            l[i] += f * ml[w].y;
#pragma unroll
            for (int b = 0; b < kCols; b += 4) {
              float y[4] = {};
              if (w > 0) get4(y, p + w * kNext + cg * 4 + b * 16);
#pragma unroll
              for (int j = 0; j < 4; j++)
                out[i][b + j] = w == 0 ? out[i][b + j] * f : fmaf(y[j], f, out[i][b + j]);
            }
          }
        }
      }
    }
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int row = warp_row + rg * 8 + i;
      const float m_scaled = m[i] * a.scale_log2;
      const int t = row / u.gp, head = u.head0 + row % u.gp;
      if (t >= u.n_tok || (few && warp > 0)) continue;
      const bool part = u.slot >= 0;
      const float inv = part ? 1.f : (l[i] == 0.f ? 0.f : 1.f / l[i]);
      const long long at = (long long)(u.row0 + t) * a.H + head;
#pragma unroll
      for (int b = 0; b < kCols; b += 4) {
        const int c = cg * 4 + b * 16;
        const float4 x = make_float4(out[i][b] * inv, out[i][b + 1] * inv, out[i][b + 2] * inv, out[i][b + 3] * inv);
        if (part) {
          a.part_o[((long long)u.slot * (D / 4) + (c >> 2)) * 64 + row] = x;
        } else {
          finite &= isfinite(x.x) && isfinite(x.y) && isfinite(x.z) && isfinite(x.w);
          *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at * D + c) = x;
        }
      }
      if (cg == 0) {
        if (part)
          a.part_ml[(long long)u.slot * 64 + row] = make_float2(m_scaled, l[i]);
        else if (a.lse)
          a.lse[at] = l[i] == 0.f ? -CUDART_INF_F : (m_scaled + log2f(l[i])) * 0.69314718056f;
      }
    }
    if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
  }
}

// Joins the pieces of the unit that block b.x of the attention kernel began
// and did not end, 32 rows per b.y, or, of many pieces of few rows, a slice of the
// columns.
// Work items are (row, four columns), 32 adjacent rows to a warp; each adds its
// pieces up in the order of the blocks that made them.  With many pieces (a
// single token over a long cache) and few rows there are more threads than items:
// they share an item's pieces.
constexpr int kMergeThreads = 512;
constexpr int kMergeRows = 32;
constexpr int kMergeUnroll = 4;
constexpr int kMergeMany = 16;  // from here on slices of columns pay (131072 keys in 64 pieces 41.5
                                // -> 35.8 us; 4 sequences of 16384 in 6 pieces each 54.8 -> 57.2)
template <class S, int D, bool BF16>
__global__ void __launch_bounds__(kMergeThreads) gdn_attn_merge_kernel(const AttnArgs a) {
  __shared__ float weight[kMergeRows], total[kMergeRows];
  __shared__ float4 part[kMergeThreads];
  __shared__ float top[kMergeRows][kMergeThreads / kMergeRows];
  const int first = blockIdx.x, tid = threadIdx.x;
  // launched while the attention kernel runs; its results are there after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const AttnJob job = a.jobs[first];
  const int n = job.last - first + 1;  // pieces
  constexpr int kSlice = D / 4 / (S::kRows / kMergeRows);  // of the columns, in fours
  const bool sliced = job.rows <= kMergeRows && n > kMergeMany;
  const int r0 = sliced ? 0 : blockIdx.y * kMergeRows;
  if (r0 >= job.rows) return;
  const int c0 = sliced ? blockIdx.y * kSlice : 0, c1 = sliced ? c0 + kSlice : D / 4;
  const int rows = min(job.rows - r0, kMergeRows);
  auto slot = [&](int i) { return (long long)(i == 0 ? 2 * first + 1 : 2 * (first + i)); };
  auto place = [&](int row) {  // of a row's head in the output
    return (long long)(job.row0 + (r0 + row) / job.gp) * a.H + job.head0 + (r0 + row) % job.gp;
  };
  bool finite = true;
  auto store = [&](int row, int d4, float4 o, float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
    const float kInf = BF16 ? kBf16Inf : CUDART_INF_F;  // from here on it is written as infinity
    finite &= fabsf(o.x) < kInf && fabsf(o.y) < kInf && fabsf(o.z) < kInf && fabsf(o.w) < kInf;
    const long long at = place(row) * D + d4 * 4;
    if constexpr (BF16) {
      __nv_bfloat162 y[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at) = *reinterpret_cast<uint2 *>(y);
    } else {
      *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) = o;
    }
  };
  auto store_lse = [&](int row, float m, float l) {
    if (a.lse && c0 == 0) a.lse[place(row)] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718056f;
  };
  // Few pieces (every unit of a call with much work): each thread reads what it
  // needs for its row at once, and none waits for another.  With the phases
  // below for these too, four prompts of 2048 tokens took 152 us cut, and 145 so;
  // two of 1023 in fp32 152 and 146.
  if (n <= kMergeUnroll) {
    const int row = tid % kMergeRows;
    if (row < rows) {
#pragma unroll 2
      for (int d4 = c0 + tid / kMergeRows; d4 < c1; d4 += kMergeThreads / kMergeRows) {
        float2 ml[kMergeUnroll];
        float4 x[kMergeUnroll];
#pragma unroll
        for (int k = 0; k < kMergeUnroll; k++) {
          const long long at = slot(k < n ? k : 0);
          ml[k] = a.part_ml[at * S::kRows + r0 + row];
          x[k] = a.part_o[(at * (D / 4) + d4) * S::kRows + r0 + row];
        }
        float m = ml[0].x, l = 0.f;
#pragma unroll
        for (int k = 1; k < kMergeUnroll; k++) m = fmaxf(m, ml[k].x);
        const float base = m == -CUDART_INF_F ? 0.f : m;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMergeUnroll; k++)
          if (k < n) {
            const float f = exp2_approx(ml[k].x - base);
            l += f * ml[k].y;
            o.x += f * x[k].x; o.y += f * x[k].y; o.z += f * x[k].z; o.w += f * x[k].w;
          }
        store(row, d4, o, l);
        if (d4 == 0) store_lse(row, m, l);
      }
    }
    if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
    return;
  }
  // row maximum and sum: kMergeThreads / 32 threads to a row
  {
    const int row = tid % kMergeRows, lane = tid / kMergeRows;
    constexpr int kLanes = kMergeThreads / kMergeRows;
    float m = -CUDART_INF_F;
    if (row < rows)
      for (int i = lane; i < n; i += kLanes)
        m = fmaxf(m, a.part_ml[slot(i) * S::kRows + r0 + row].x);
    top[row][lane] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLanes; i++) m = fmaxf(m, top[row][i]);
    const float base = m == -CUDART_INF_F ? 0.f : m;
    float l = 0.f;
    if (row < rows)
      for (int i = lane; i < n; i += kLanes) {
        const float2 ml = a.part_ml[slot(i) * S::kRows + r0 + row];
        l += exp2_approx(ml.x - base) * ml.y;
      }
    __syncthreads();
    top[row][lane] = l;
    __syncthreads();
    if (lane == 0 && row < rows) {
      l = 0.f;
      for (int i = 0; i < kLanes; i++) l += top[row][i];
      weight[row] = base;
      total[row] = l;
      store_lse(row, m, l);
    }
    __syncthreads();
  }
  // rows rounded up to a power of two, so that a warp's threads have adjacent rows
  int wide = 1;
  while (wide < rows) wide <<= 1;
  const int items = wide * (c1 - c0);
  const int share = items >= kMergeThreads ? 1 : kMergeThreads / items;  // threads to an item
  for (int i0 = 0; i0 < items; i0 += kMergeThreads / share) {
    const int item = i0 + tid % (kMergeThreads / share), who = tid / (kMergeThreads / share);
    const int row = item % wide, d4 = c0 + item / wide;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows) {
      const float base = weight[row];
      for (int i = who * kMergeUnroll; i < n; i += share * kMergeUnroll) {
        float4 x[kMergeUnroll];
        float f[kMergeUnroll];
#pragma unroll
        for (int k = 0; k < kMergeUnroll; k++) {
          const bool have = i + k < n;
          const long long at = slot(have ? i + k : 0);
          f[k] = have ? exp2_approx(a.part_ml[at * S::kRows + r0 + row].x - base) : 0.f;
          x[k] = a.part_o[(at * (D / 4) + d4) * S::kRows + r0 + row];
        }
#pragma unroll
        for (int k = 0; k < kMergeUnroll; k++)
          if (i + k < n) {
            o.x += f[k] * x[k].x; o.y += f[k] * x[k].y; o.z += f[k] * x[k].z; o.w += f[k] * x[k].w;
          }
      }
    }
    if (share > 1) {
      part[tid] = o;
      __syncthreads();
      if (who == 0)
        for (int w = 1; w < share; w++) {
          const float4 x = part[tid + w * (kMergeThreads / share)];
          o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
        }
      __syncthreads();
    }
    if (row >= rows || who != 0) continue;
    store(row, d4, o, total[row]);
  }
  if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
}

template <class S, int D, bool BF16>
cudaError_t merge(const AttnArgs &a, int blocks, cudaStream_t stream) {
  // may be set up while the attention kernel still runs
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(blocks - 1, S::kRows / kMergeRows);
  config.blockDim = dim3(kMergeThreads);
  config.stream = stream;
  config.attrs = &early;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, gdn_attn_merge_kernel<S, D, BF16>, a);
}

template <int D>
std::atomic<uint64_t> allowed{0};

template <int D>
cudaError_t launch(const AttnArgs &a, int blocks, cudaStream_t stream) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void *>(&gdn_attn_warp_kernel<D>),
                                   WarpSmem<D>::kBytes, allowed<D>);
  if (e != cudaSuccess) return e;
  gdn_attn_warp_kernel<D><<<blocks, kThreads, WarpSmem<D>::kBytes, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
      if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
      return n;
    }
  }
  (void)cudaGetLastError();  // no device: sizes can still be asked for
  return 152;
}

cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

AttnLaunch attn_launch(AttnArgs &a, int d, int dtype) {
  return dtype ? attn_plan_launch<TcShape>(a, sm_count())
               : attn_plan_launch<WarpShape>(a, sm_count() * (d == 64 ? blocks_per_sm<64>() : blocks_per_sm<128>()));
}

cudaError_t launch_attn(const AttnArgs &a, int d, int dtype, const AttnLaunch &l,
                        cudaStream_t stream) {
  cudaError_t e;
  if (dtype)
    e = launch_attn_tc(a, d, l.blocks, stream);
  else
    e = d == 64 ? launch<64>(a, l.blocks, stream) : launch<128>(a, l.blocks, stream);
  if (e != cudaSuccess || !l.split || l.blocks < 2) return e;
  if (dtype)
    return d == 64 ? merge<TcShape, 64, true>(a, l.blocks, stream)
                   : merge<TcShape, 128, true>(a, l.blocks, stream);
  return d == 64 ? merge<WarpShape, 64, false>(a, l.blocks, stream)
                 : merge<WarpShape, 128, false>(a, l.blocks, stream);
}

}  // namespace gdn
