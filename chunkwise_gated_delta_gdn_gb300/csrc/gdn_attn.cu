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

#include "gdn_attn.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace {

// fp32: 64 rows x 64 keys per step: four warps of 16 rows, the operands in shared
// memory as fp32, both products split-tf32 on mma.sync.
using WarpShape = AttnShape<64, 64, 64, 1, 1>;
using TcShape = AttnShape<256, 128, 128, 2, 4>;  // of the bf16 kernel (gdn_attn_tc.cu)
constexpr int kThreads = 128;

template <int D>
constexpr int smem_bytes() { return 3 * 64 * (D + 4) * 4; }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c += A B for one 16 x 8 tile, k = 8: the three products of the two halves
__device__ __forceinline__ void mma3(float (&c)[4], const uint32_t (&ah)[4],
                                     const uint32_t (&al)[4], float b0, float b1) {
  uint32_t h0, l0, h1, l1;
  split_tf32(b0, h0, l0);
  split_tf32(b1, h1, l1);
  mma1688_tf32(c, al, h0, h1);
  mma1688_tf32(c, ah, l0, l1);
  mma1688_tf32(c, ah, h0, h1);
}

__device__ __forceinline__ void load8(float (&x)[8], const float *p) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
  const float4 b = __ldg(reinterpret_cast<const float4 *>(p + 4));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void put8(float *d, const float (&x)[8]) {
  *reinterpret_cast<float4 *>(d) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4 *>(d + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) gdn_attn_warp_kernel(const AttnArgs a) {
  constexpr int kS = D + 4;  // row stride in floats: fragment reads hit 32 banks
  extern __shared__ float smem[];
  float *Qs = smem, *Ks = Qs + 64 * kS, *Vs = Ks + 64 * kS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, tq = lane & 3;
  AttnPlan<WarpShape> plan(a.H, a.HKV, a.plan_coarse);
  AttnStaged *staged = reinterpret_cast<AttnStaged *>(smem);  // until the first operands
  attn_stage(a, staged, blockIdx.x);
  __syncthreads();
  const AttnStart st = attn_start(a, plan, staged, blockIdx.x, gridDim.x);  // each warp for itself
  AttnWalk<WarpShape> walk(a, plan, st, blockIdx.x);
  AttnUnit u;
  if (a.jobs && tid == 0) a.jobs[blockIdx.x].rows = 0;
  while (walk.next(u)) {
    if (tid == 0 && u.slot == 2 * (int)blockIdx.x + 1) a.jobs[blockIdx.x] = attn_job(u);
    __syncthreads();  // the previous unit's operands (or the plan's) are read
    for (int i = tid; i < 64 * (D / 8); i += kThreads) {
      const int r = i / (D / 8), c = (i % (D / 8)) * 8, t = r / u.gp;
      float x[8] = {};
      if (t < u.n_tok)
        load8(x, static_cast<const float *>(a.q) + (long long)(u.row0 + t) * a.q_stride +
                           (u.head0 + r % u.gp) * D + c);
      put8(Qs + r * kS + c, x);
    }
    float o[D / 8][4] = {}, m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    const int row[2] = {warp * 16 + gq, warp * 16 + gq + 8};
    int limit[2];  // last visible key
#pragma unroll
    for (int h = 0; h < 2; h++) limit[h] = min(u.pos0 + row[h] / u.gp, u.len - 1);
    for (int t = u.t0; t < u.t1; t++) {
      const int key0 = t * 64;
      __syncthreads();
      for (int i = tid; i < 2 * 64 * (D / 8); i += kThreads) {
        const bool is_v = i >= 64 * (D / 8);
        const int j = is_v ? i - 64 * (D / 8) : i, r = j / (D / 8), c = (j % (D / 8)) * 8;
        const int key = key0 + r;
        float x[8] = {};
        if (key < u.len) {
          const float *p = static_cast<const float *>(is_v ? a.v : a.k);
          bool ok = true;
          if (a.table) {
            const int page = __ldg(a.table + (long long)u.seq * a.max_pages + key / a.page_size);
            ok = page >= 0 && page < a.n_pages;
            if (!ok && a.flags) atomicOr(a.flags, kFlagBadSeqlens);
            p += (((long long)page * a.page_size + key % a.page_size) * a.HKV + u.kvh) * D;
          } else {
            // a prompt's keys are its own tokens
            p += (long long)(u.row0 - u.pos0 + key) * (is_v ? a.v_stride : a.k_stride) + u.kvh * D;
          }
          if (ok) load8(x, p + c);
        }
        put8((is_v ? Vs : Ks) + r * kS + c, x);
      }
      __syncthreads();
      float s[8][4] = {};
#pragma unroll 4
      for (int k = 0; k < D; k += 8) {
        uint32_t ah[4], al[4];
        const float *q0 = Qs + row[0] * kS + k + tq, *q1 = Qs + row[1] * kS + k + tq;
        split_tf32(q0[0], ah[0], al[0]);
        split_tf32(q1[0], ah[1], al[1]);
        split_tf32(q0[4], ah[2], al[2]);
        split_tf32(q1[4], ah[3], al[3]);
#pragma unroll
        for (int n = 0; n < 8; n++) {
          const float *b = Ks + (n * 8 + gq) * kS + k + tq;
          mma3(s[n], ah, al, b[0], b[4]);
        }
      }
      // running maximum and sum; element e of a tile: row e / 2, key 2 tq + e % 2
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float top = m[h];
#pragma unroll
        for (int n = 0; n < 8; n++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float &x = s[n][2 * h + e];
            x = key0 + n * 8 + 2 * tq + e <= limit[h] ? x * a.scale_log2 : -CUDART_INF_F;
            top = fmaxf(top, x);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float base = top == -CUDART_INF_F ? 0.f : top;  // nothing visible yet
        const float alpha = exp2_approx(m[h] - base);
        m[h] = top;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 8; n++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float &x = s[n][2 * h + e];
            x = exp2_approx(x - base);
            sum += x;
          }
        l[h] = l[h] * alpha + sum;
#pragma unroll
        for (int n = 0; n < D / 8; n++) {
          o[n][2 * h] *= alpha;
          o[n][2 * h + 1] *= alpha;
        }
      }
      // the weights are the A operand as they lie: contraction index tq stands
      // for key 2 tq, index tq + 4 for key 2 tq + 1
#pragma unroll
      for (int n = 0; n < 8; n++) {
        uint32_t ah[4], al[4];
        split_tf32(s[n][0], ah[0], al[0]);
        split_tf32(s[n][2], ah[1], al[1]);
        split_tf32(s[n][1], ah[2], al[2]);
        split_tf32(s[n][3], ah[3], al[3]);
        const float *b = Vs + (n * 8 + 2 * tq) * kS + gq;
#pragma unroll
        for (int d = 0; d < D / 8; d++) mma3(o[d], ah, al, b[d * 8], b[kS + d * 8]);
      }
    }
    bool finite = true;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      const int t = row[h] / u.gp, head = u.head0 + row[h] % u.gp;
      if (t >= u.n_tok) continue;
      if (u.slot >= 0) {
        float2 *po = reinterpret_cast<float2 *>(a.part_o + (long long)u.slot * 64 * (D / 4));
#pragma unroll
        for (int n = 0; n < D / 8; n++)  // columns n*8 + 2 tq: half of float4 n*2 + tq/2
          po[((long long)(n * 2 + (tq >> 1)) * 64 + row[h]) * 2 + (tq & 1)] =
              make_float2(o[n][2 * h], o[n][2 * h + 1]);
        if (tq == 0) a.part_ml[(long long)u.slot * 64 + row[h]] = make_float2(m[h], l[h]);
        continue;
      }
      const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
      const long long at = (long long)(u.row0 + t) * a.H + head;
#pragma unroll
      for (int n = 0; n < D / 8; n++) {
        const float x = o[n][2 * h] * inv, y = o[n][2 * h + 1] * inv;
        finite &= isfinite(x) && isfinite(y);
        *reinterpret_cast<float2 *>(static_cast<float *>(a.o) + at * D + n * 8 + 2 * tq) =
            make_float2(x, y);
      }
      if (a.lse && tq == 0) a.lse[at] = l[h] == 0.f ? -CUDART_INF_F : (m[h] + log2f(l[h])) * 0.69314718056f;
    }
    if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
  }
}

// Joins the pieces of the unit that block b.x of the attention kernel began
// and did not end, 32 rows per b.y.  Work items are (row, four columns), 32
// adjacent rows to a warp; each adds its pieces up in the order of the blocks
// that made them.  With many pieces (a single token over a long cache) and few
// rows there are more threads than items: they share an item's pieces.
constexpr int kMergeThreads = 512;
constexpr int kMergeRows = 32;
constexpr int kMergeUnroll = 4;
template <class S, int D, bool BF16>
__global__ void __launch_bounds__(kMergeThreads) gdn_attn_merge_kernel(const AttnArgs a) {
  __shared__ float weight[kMergeRows], total[kMergeRows];
  __shared__ float4 part[kMergeThreads];
  __shared__ float top[kMergeRows][kMergeThreads / kMergeRows];
  const int first = blockIdx.x, r0 = blockIdx.y * kMergeRows, tid = threadIdx.x;
  // launched while the attention kernel runs; its results are there after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const AttnJob job = a.jobs[first];
  if (r0 >= job.rows) return;
  const int n = job.last - first + 1;  // pieces
  const int rows = min(job.rows - r0, kMergeRows);
  auto slot = [&](int i) { return (long long)(i == 0 ? 2 * first + 1 : 2 * (first + i)); };
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
      if (a.lse) {
        const long long at = (long long)(job.row0 + (r0 + row) / job.gp) * a.H + job.head0 + (r0 + row) % job.gp;
        a.lse[at] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718056f;
      }
    }
    __syncthreads();
  }
  // rows rounded up to a power of two, so that a warp's threads have adjacent rows
  int wide = 1;
  while (wide < rows) wide <<= 1;
  const int items = wide * (D / 4);
  const int share = items >= kMergeThreads ? 1 : kMergeThreads / items;  // threads to an item
  bool finite = true;
  for (int i0 = 0; i0 < items; i0 += kMergeThreads / share) {
    const int item = i0 + tid % (kMergeThreads / share), who = tid / (kMergeThreads / share);
    const int row = item % wide, d4 = item / wide;
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
    const float inv = total[row] == 0.f ? 0.f : 1.f / total[row];
    o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
    finite &= isfinite(o.x) && isfinite(o.y) && isfinite(o.z) && isfinite(o.w);
    const long long at = (long long)(job.row0 + (r0 + row) / job.gp) * a.H + job.head0 + (r0 + row) % job.gp;
    if constexpr (BF16) {
      __nv_bfloat162 y[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + d4 * 4) =
          *reinterpret_cast<uint2 *>(y);
    } else {
      *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at * D + d4 * 4) = o;
    }
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
                                   smem_bytes<D>(), allowed<D>);
  if (e != cudaSuccess) return e;
  gdn_attn_warp_kernel<D><<<blocks, kThreads, smem_bytes<D>(), stream>>>(a);
  return cudaGetLastError();
}

template <class S>
AttnLaunch plan_launch(AttnArgs &a, int blocks) {
  AttnLaunch l;
  l.blocks = blocks;
  l.rows = S::kRows;
  a.plan_total = 0;
  // Nothing is cut when every unit fits the smallest grain and gets a block.
  const long long units = attn_most_units<S>(a);
  const int longest = a.kv_lens ? a.max_len : (a.cu ? a.Ttot : a.T);
  l.split = !(AttnPlan<S>::tiles(longest) <= 1 << kMinGrain && units <= blocks);
  if (!l.split) l.blocks = units < 1 ? 1 : (int)units;
  a.plan_coarse = attn_coarse<S>(units, longest);
  if (a.plan_coarse < 0) {
    l.blocks = 0;
    return l;
  }
  if (!a.cu && !a.kv_lens && a.T > 0) l.split = attn_plan_prompts<S>(a, l.blocks);
  return l;
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
  return dtype ? plan_launch<TcShape>(a, sm_count())
               : plan_launch<WarpShape>(a, sm_count() * (d == 64 ? 4 : 2));
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
