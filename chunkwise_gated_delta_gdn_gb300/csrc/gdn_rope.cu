// gdn_rope.cu -- rotary positions: pairs (a, b) of the first `rot` elements of each
// query and key head are turned by the angle p f_i of their token's position p and
// their frequency f_i,
//   a' = mscale (a cos - b sin),  b' = mscale (a sin + b cos),
// pair i being elements (i, i + rot / 2) or, interleaved, (2 i, 2 i + 1); the rest of
// a head is copied.  Backward: the same with -sin (the transpose).
//
// A far position's angle has to be exact modulo a turn: p f in fp32 is off by 2^-7 at
// 131072.  So, as in the published reduction of large arguments by a long 1 / 2 pi (Payne and
// Hanek), f / 2 pi is taken as a 64-bit fraction of a turn in integer arithmetic
// (fp64 is slow here), times p modulo 2^64: whole turns fall away, and what is left is
// off by less than 2^-33 of a turn from f's places cut off (32-bit positions) and 2^-32 from those
// of the product.  The rest, at most 1/8 of a turn, is then taken to fp32, which adds 2^-28
// of a turn at most: 2^-25.2 in all.
//
// Bound by memory.  A block turns a few tokens: their sines and cosines once, into
// shared memory, for all heads; then each thread takes two 16-byte pieces, those that
// hold the two elements of its pairs, the next ones on their way meanwhile (the first
// while the angles are made; two ahead took registers and time).  q and k of 32768
// tokens, 32/8 heads of 128: 105 us, 6.4 TB/s read and written; 12001 tokens of 16/16 heads of
// 64 in fp32: 33 us; 256 sequences of one token: 3.3 us.
#include <cuda_bf16.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // of a block
constexpr int kItemsWanted = 2560;  // of a block: ten for each thread

// f / 2 pi modulo 1, in 2^-64 (less than one of them too small in magnitude), for f
// finite and below 2^63: the mantissa of f, an integer, times the 128 binary places of
// 1 / 2 pi from 32 behind the last that matters on.
__device__ __forceinline__ uint64_t turns_of(float f) {
  const uint32_t b = __float_as_uint(f);
  const int e = b >> 23 & 255, k = (e ? e : 1) - 54;  // f = mantissa 2^(k - 96)
  if (k <= 0 || k > 135) return 0;                    // nothing left at 2^-64 (or out of range)
  // 1 / 2 pi = 0x0.28be60db 9391054a 7f09d5f4 7d4d3770 36d8a566 4f10e410 ..
  const uint64_t places[5] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull, 0, 0};
  const int down = 192 - k, bit = down & 63;
  uint64_t w[3];
#pragma unroll
  for (int i = 0; i < 3; i++) {
    w[i] = places[i];
    if (down >= 128) w[i] = places[i + 2];
    else if (down >= 64) w[i] = places[i + 1];
  }
  unsigned __int128 window = (unsigned __int128)w[1] << 64 | w[0];
  if (bit) window = window >> bit | (unsigned __int128)w[2] << (128 - bit);
  const uint64_t mant = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
  const uint64_t t = (uint64_t)(window * mant >> 32);
  return b >> 31 ? 0 - t : t;
}

// Sequence of token row t and the row's position; false when it belongs to none that
// is well formed.
__device__ __forceinline__ bool position(const RopeArgs &a, int t, int &pos) {
  int n, start, end;
  if (a.cu) {
    int lo = 0, hi = a.n_seqs - 1;  // the last n with cu[n] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid - 1;
    }
    n = lo;
    start = __ldg(a.cu + n);
    end = __ldg(a.cu + n + 1);
  } else {
    n = t / a.T;
    start = n * a.T;
    end = start + a.T;
  }
  const int nq = end - start, len = a.kv_lens ? __ldg(a.kv_lens + n) : nq;
  pos = len - nq + (t - start);
  return start >= 0 && start <= t && t < end && end <= a.Ttot && len >= 0;
}

template <typename T>
struct Piece;  // 16 bytes
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4 &w, float (&x)[8]) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[2 * i] = __uint_as_float(ws[i] << 16);
      x[2 * i + 1] = __uint_as_float(ws[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    uint32_t ws[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      ws[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(ws[0], ws[1], ws[2], ws[3]);
  }
};
template <>
struct Piece<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4 &w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) gdn_rope_kernel(const RopeArgs a, const int tokens) {
  using P = Piece<T>;
  constexpr int kN = P::kN, kItems = D / (2 * kN);  // of a head
  __shared__ float2 turn[kMaxTokens][D / 2];  // (cos, sin)
  __shared__ int place[kMaxTokens];           // positions
  __shared__ bool valid[kMaxTokens];
  const int first = blockIdx.x * tokens, here = min(tokens, a.Ttot - first);
  const int pairs = a.rot / 2, heads = a.HQ + a.HK, items = here * heads * kItems;
  // The two pieces of item i: their first elements, where they are read and written.
  struct Item {
    int tok, e0, e1;
    const T *x;
    T *y;
  };
  auto item = [&](int i) {
    const int j = i % kItems, row = i / kItems, tok = row / heads, head = row - tok * heads;
    const bool is_q = head < a.HQ;
    const long long at = first + tok;
    Item r;
    r.tok = tok;
    r.x = is_q ? static_cast<const T *>(a.q) + at * a.q_stride + head * D
               : static_cast<const T *>(a.k) + at * a.k_stride + (head - a.HQ) * D;
    r.y = is_q ? static_cast<T *>(a.qo) + at * a.qo_stride + head * D
               : static_cast<T *>(a.ko) + at * a.ko_stride + (head - a.HQ) * D;
    const int turned = pairs / kN;  // items that are turned, where halves are paired
    if (INTERLEAVED || j >= turned) {
      r.e0 = INTERLEAVED ? 2 * j * kN : 2 * pairs + 2 * (j - turned) * kN;
      r.e1 = r.e0 + kN;
    } else {
      r.e0 = j * kN;
      r.e1 = pairs + r.e0;
    }
    return r;
  };
  // The first item's pieces are on their way while the angles are made.
  Item next = item(min((int)threadIdx.x, items - 1));
  uint4 n0 = *reinterpret_cast<const uint4 *>(next.x + next.e0), n1 = *reinterpret_cast<const uint4 *>(next.x + next.e1);
  // A token finds its sequence by halving, and so need not meet a malformed one.
  if (a.cu && a.flags)
    for (long long n = (long long)blockIdx.x * kThreads + threadIdx.x; n < a.n_seqs; n += (long long)gridDim.x * kThreads) {
      const int from = __ldg(a.cu + n), to = __ldg(a.cu + n + 1);
      if (from < 0 || to < from || to > a.Ttot) atomicOr(a.flags, kFlagBadSeqlens);
    }
  if (threadIdx.x < here) {
    int pos;
    const bool ok = position(a, first + threadIdx.x, pos);
    place[threadIdx.x] = pos;
    valid[threadIdx.x] = ok;
    if (!ok && a.flags) atomicOr(a.flags, kFlagBadSeqlens);
  }
  // A thread has a pair of every few tokens.
  const int apart = kThreads / pairs, pair = threadIdx.x % pairs, tok0 = threadIdx.x / pairs;
  const uint64_t t = turns_of(__ldg(a.inv_freq + pair));
  __syncthreads();
  for (int tok = tok0; tok < here && tok0 < apart; tok += apart) {
    // the angle in 2^-32 turns: a quarter, and the rest from -1/8 to 1/8
    const uint32_t angle = (uint32_t)(((uint64_t)(int64_t)place[tok] * t) >> 32);
    const uint32_t quarter = (angle + 0x20000000u) >> 30;
    float s, c;
    sincospif((float)(int)(angle - (quarter << 30)) * 0x1p-31f, &s, &c);
    const float qs = quarter & 1 ? c : s, qc = quarter & 1 ? s : c;
    turn[tok][pair] = make_float2((quarter + 1) & 2 ? -qc * a.mscale : qc * a.mscale,
                                  (quarter & 2 ? -qs : qs) * a.mscale * a.sign);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const Item r = next;
    const uint4 w0 = n0, w1 = n1;
    if (i + kThreads < items) {
      next = item(i + kThreads);
      n0 = *reinterpret_cast<const uint4 *>(next.x + next.e0);
      n1 = *reinterpret_cast<const uint4 *>(next.x + next.e1);
    }
    if (!valid[r.tok]) continue;
    uint4 z0 = w0, z1 = w1;
    if (r.e0 < a.rot) {
      float u[kN], v[kN], p[kN], q[kN];
      P::get(w0, u);
      P::get(w1, v);
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int k = 0; k < kN; k += 2) {
          const float2 c0 = turn[r.tok][(r.e0 + k) / 2], c1 = turn[r.tok][(r.e1 + k) / 2];
          p[k] = u[k] * c0.x - u[k + 1] * c0.y;
          p[k + 1] = u[k] * c0.y + u[k + 1] * c0.x;
          q[k] = v[k] * c1.x - v[k + 1] * c1.y;
          q[k + 1] = v[k] * c1.y + v[k + 1] * c1.x;
        }
      } else {
#pragma unroll
        for (int k = 0; k < kN; k++) {
          const float2 c = turn[r.tok][r.e0 + k];
          p[k] = u[k] * c.x - v[k] * c.y;
          q[k] = u[k] * c.y + v[k] * c.x;
        }
      }
      z0 = P::put(p);
      z1 = P::put(q);
    }
    *reinterpret_cast<uint4 *>(r.y + r.e0) = z0;
    *reinterpret_cast<uint4 *>(r.y + r.e1) = z1;
  }
}

template <typename T, int D>
cudaError_t launch(const RopeArgs &a, bool interleaved, cudaStream_t stream) {
  // several tokens to a block where they have few heads and every SM has blocks enough
  const int items = (a.HQ + a.HK) * D / (2 * Piece<T>::kN), most = a.Ttot / (4 * sm_count());
  int tokens = kItemsWanted / items;
  if (tokens > most) tokens = most;
  if (tokens > kMaxTokens) tokens = kMaxTokens;
  if (tokens < 1) tokens = 1;
  const unsigned blocks = (unsigned)((a.Ttot + tokens - 1) / tokens);
  if (interleaved) gdn_rope_kernel<T, D, true><<<blocks, kThreads, 0, stream>>>(a, tokens);
  else gdn_rope_kernel<T, D, false><<<blocks, kThreads, 0, stream>>>(a, tokens);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int d, bool interleaved, int dtype, cudaStream_t stream) {
  if (dtype) return d == 64 ? launch<__nv_bfloat16, 64>(a, interleaved, stream) : launch<__nv_bfloat16, 128>(a, interleaved, stream);
  return d == 64 ? launch<float, 64>(a, interleaved, stream) : launch<float, 128>(a, interleaved, stream);
}

}  // namespace gdn
