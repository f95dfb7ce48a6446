// gdn_kv_append8.cu -- writes the keys and values of new tokens into the pages
// of a cache held in 8 bits (e4m3 values, an fp32 scale for each block of 16
// tokens and head).  Of a block that new tokens reach,
//   need = the smallest power of two, 2^-117 or more, with max |new| <= 448 need,
//   a' = need, or max(a, need) where the block holds earlier tokens (scale a),
//   held values c -> round(c a / a'), new ones x -> round(x / a'),
// to the nearest e4m3 value, ties to even; a non-finite x becomes NaN.  Powers of
// two make both exact but for that rounding, and a held value is rounded again only
// where it falls below 2^-6 a'.
//
// A warp has a block of one head, keys or values: 16 rows, eight elements of a row
// to a lane.  A copy by its cost: bound by memory, and by launch and three reads in a
// row (length, page, scale) for a decode step.  32768 tokens of 8 heads of 128: 31.5 us,
// 6.4 TB/s read and written (120 us where each row's read was waited for before the
// next one's; 34.5 with 24 warps to an SM in blocks of eight, 32.8 in blocks of four, so
// 32 warps); 256 sequences of one token: 4.2 us.
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kWarps = 4;

// all lanes: the last n with at(n) <= x, at non-decreasing and at(0) <= x
template <class F>
__device__ __forceinline__ int last_at(F at, int n_seqs, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, n = min(lo + (lane + 1) * step, hi);
    const int below = __popc(__ballot_sync(0xffffffffu, at(n) <= x));  // of non-decreasing ones: the first `below`
    const int next = min(lo + below * step, hi);
    hi = min(hi, max(next, next + step - 1));
    lo = next;
    if (below == 32) break;
  }
  return lo;
}

// four fp32 values as four e4m3 in a word
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ void from_e4m3(uint32_t x, float (&y)[4]) {
  asm("{\n .reg .b16 l, h, a, b, c, d;\n .reg .b32 p, q;\n mov.b32 {l, h}, %4;\n cvt.rn.f16x2.e4m3x2 p, l;\n cvt.rn.f16x2.e4m3x2 q, h;\n"
      " mov.b32 {a, b}, p;\n mov.b32 {c, d}, q;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n cvt.f32.f16 %2, c;\n cvt.f32.f16 %3, d;\n}"
      : "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3])
      : "r"(x));
}

// Eight elements of a row, as they came, and as numbers.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ void get(const void *p) { w = __ldg(static_cast<const uint4 *>(p)); }
  __device__ void zero() { w = make_uint4(0, 0, 0, 0); }
  // the largest magnitude, as the bits of an fp32 number
  __device__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
    return max(t << 16, t & 0x7fff0000u);
  }
  __device__ void put(float (&y)[8]) const {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
      y[2 * e] = __uint_as_float(ws[e] << 16);
      y[2 * e + 1] = __uint_as_float(ws[e] & 0xffff0000u);
    }
  }
};
template <>
struct Eight<float> {
  float4 u, w;
  __device__ void get(const void *p) {
    u = __ldg(static_cast<const float4 *>(p));
    w = __ldg(static_cast<const float4 *>(p) + 1);
  }
  __device__ void zero() { u = w = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ uint32_t top() const {
    float y[8];
    put(y);
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) t = max(t, __float_as_uint(y[e]) & 0x7fffffffu);
    return t;
  }
  __device__ void put(float (&y)[8]) const {
    y[0] = u.x; y[1] = u.y; y[2] = u.z; y[3] = u.w;
    y[4] = w.x; y[5] = w.y; y[6] = w.z; y[7] = w.w;
  }
};

// A block of warps has the heads, keys and values, of a slot (of a block of tokens),
// several blocks where there are more than kWarps of them.
template <int D, typename T>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 8 : 4) gdn_kv_append8_kernel(const Append8Args a, const int per_seq) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kPasses = kScaleBlock / kAtOnce;
  const int lane = threadIdx.x & 31;
  if (a.cu && a.flags && blockIdx.y == 0)  // a slot finds its sequence, and so need not meet a malformed one
    for (long long n = (long long)blockIdx.x * blockDim.x + threadIdx.x; n < a.n_seqs; n += (long long)gridDim.x * blockDim.x) {
      const int from = __ldg(a.cu + n), to = __ldg(a.cu + n + 1);
      if (from < 0 || to < from || to > a.Ttot) atomicOr(a.flags, kFlagBadSeqlens);
    }
  const int slot = blockIdx.x, rest = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (rest >= 2 * a.HKV) return;
  const int head = rest >> 1, which = rest & 1;  // keys (0) or values (1)
  // Sequence n has per_seq slots, or, packed, those from floor(cu[n] / 16) + 2 n on: it
  // reaches at most floor((nq + 30) / 16) blocks.
  int n, start, end, j;
  if (a.cu) {
    n = last_at([&](int i) { return __ldg(a.cu + i) / kScaleBlock + 2 * i; }, a.n_seqs, slot);
    start = __ldg(a.cu + n);
    end = __ldg(a.cu + n + 1);
    if (start < 0 || end < start || end > a.Ttot) return;  // reported above
    j = slot - start / kScaleBlock - 2 * n;
    if (j < 0) return;
  } else {
    n = per_seq == 1 ? slot : slot / per_seq;
    j = slot - n * per_seq;
    start = n * a.T;
    end = start + a.T;
  }
  const int len = __ldg(a.kv_lens + n), past = len - (end - start);
  if (len < 0 || len > a.max_len) {
    if (a.flags && lane == 0) atomicOr(a.flags, kFlagBadSeqlens);
    return;
  }
  // the block's first position
  const long long p0 = ((long long)(max(past, 0) / kScaleBlock) + j) * kScaleBlock;
  if (p0 >= len || end == start) return;
  const int pos0 = (int)p0, place = pos0 / a.page_size, inside = pos0 - place * a.page_size;
  const int page = __ldg(a.table + (long long)n * a.max_pages + place);
  const int row = lane / kLanes, col = lane % kLanes * 8;
  // All rows' reads are on their way before anything waits for one.
  Eight<T> x[kPasses];
  {
    const T *from = static_cast<const T *>(which ? a.v : a.k) + head * D + col;
    const long long stride = which ? a.v_stride : a.k_stride;
#pragma unroll
    for (int i = 0; i < kPasses; i++) {
      const int pos = pos0 + i * kAtOnce + row;
      x[i].zero();
      if (pos >= past && pos < len) x[i].get(from + (long long)(start + (pos - past)) * stride);
    }
  }
  if (page < 0 || page >= a.n_pages) {
    if (a.flags && lane == 0) atomicOr(a.flags, kFlagBadSeqlens);
    return;
  }
  float *scale_at = (which ? a.v_scale : a.k_scale) + ((long long)page * (a.page_size / kScaleBlock) + inside / kScaleBlock) * a.HKV + head;
  const bool holds = pos0 < past;
  const float held = holds ? *scale_at : 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPasses; i++) top = max(top, x[i].top());
  top = __reduce_max_sync(0xffffffffu, top);
  const bool odd = top >= 0x7f800000u;  // something is not finite: it becomes NaN and does not count for the scale
  if (odd) {
    top = 0;
#pragma unroll 1
    for (int i = 0; i < kPasses; i++) {
      float y[8];
      x[0].put(y);
#pragma unroll
      for (int k = 1; k < kPasses; k++)
        if (k == i) x[k].put(y);
#pragma unroll
      for (int c = 0; c < 8; c++)
        if (isfinite(y[c])) top = max(top, __float_as_uint(y[c]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (a.flags && lane == 0) atomicOr(a.flags, kFlagNonfinite);
  }
  // top = f 2^k with f in [1, 2): top <= 1.75 2^8 2^e
  const int e = top == 0 ? -117 : min(max((int)((top + 0x1fffffu) >> 23) - 135, -117), 120);
  const float need = __int_as_float((127 + e) << 23), scale = fmaxf(held, need);
  uint8_t *cache = (which ? a.v_cache : a.k_cache) + (((long long)page * a.page_size + inside) * a.HKV + head) * D + col;
  const long long cache_row = (long long)a.HKV * D;
  auto write = [&](auto quotient) {
#pragma unroll
    for (int i = 0; i < kPasses; i++) {
      const int r = i * kAtOnce + row, pos = pos0 + r;
      float y[8];
      x[i].put(y);
      const uint2 z = make_uint2(to_e4m3(quotient(y[0]), quotient(y[1]), quotient(y[2]), quotient(y[3])),
                                 to_e4m3(quotient(y[4]), quotient(y[5]), quotient(y[6]), quotient(y[7])));
      if (pos >= past && pos < len) *reinterpret_cast<uint2 *>(cache + r * cache_row) = z;
    }
  };
  const bool power = (__float_as_uint(scale) & 0x7fffffu) == 0 && scale < 0x1p127f;
  if (power && !odd) {
    const float inv = __int_as_float((254 << 23) - __float_as_int(scale));  // 1 / scale, exact
    write([&](float y) { return y * inv; });
  } else {
    write([&](float y) { return isfinite(y) ? __fdiv_rn(y, scale) : CUDART_NAN_F; });
  }
  if (!(scale > held)) return;
  if (holds) {
    const float down = __fdiv_rn(held, scale);
#pragma unroll
    for (int i = 0; i < kPasses; i++) {
      const int r = i * kAtOnce + row;
      if (pos0 + r >= past) continue;
      uint2 *at = reinterpret_cast<uint2 *>(cache + r * cache_row);
      const uint2 w = *at;
      float lo[4], hi[4];
      from_e4m3(w.x, lo);
      from_e4m3(w.y, hi);
#pragma unroll
      for (int c = 0; c < 4; c++) {
        lo[c] = __fmul_rn(lo[c], down);
        hi[c] = __fmul_rn(hi[c], down);
      }
      *at = make_uint2(to_e4m3(lo[0], lo[1], lo[2], lo[3]), to_e4m3(hi[0], hi[1], hi[2], hi[3]));
    }
  }
  __syncwarp();  // every lane has read the held scale
  if (lane == 0) *scale_at = scale;
}

template <int D, typename T>
cudaError_t launch(const Append8Args &a, cudaStream_t stream) {
  const int per_seq = (int)(((long long)a.T + 2 * kScaleBlock - 2) / kScaleBlock);
  const long long slots = a.cu ? a.Ttot / kScaleBlock + 2LL * a.n_seqs : (long long)a.n_seqs * per_seq;
  const int warps = 2 * a.HKV < kWarps ? 2 * a.HKV : kWarps;
  if (slots > INT32_MAX) return cudaErrorInvalidValue;
  gdn_kv_append8_kernel<D, T><<<dim3((unsigned)slots, (2 * a.HKV + warps - 1) / warps), warps * 32, 0, stream>>>(a, per_seq);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append8(const Append8Args &a, int d, int dtype, cudaStream_t stream) {
  if (dtype) return d == 64 ? launch<64, __nv_bfloat16>(a, stream) : launch<128, __nv_bfloat16>(a, stream);
  return d == 64 ? launch<64, float>(a, stream) : launch<128, float>(a, stream);
}

}  // namespace gdn
