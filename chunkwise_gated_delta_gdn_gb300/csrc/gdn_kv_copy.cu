// gdn_kv_copy.cu -- copies whole pages of a cache: page src[i] to page dst[i], keys,
// values and, of a cache in 8 bits, scales, as when a sequence forks (its last page,
// which both go on writing) or a pool is put in order.
//
// Every pair reads what was there before the call: a page that is the destination of
// two pairs, or of one and the source of another, is left as it is, and reported.  A
// block looks that up for the pairs that it copies, kOwn at a time, while it goes
// through all pairs once: n^2 / blocks comparisons, 108 for each thread with 4096 pairs.
//
// A copy, bound by memory: 16 bytes to a thread, four in flight; a pair is split
// between blocks while there are fewer pairs than the SMs want.
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 512;
constexpr int kOwn = 32;

__device__ __forceinline__ void copy(char *to, const char *from, long long bytes, int part, int parts) {
  if (((uintptr_t)to | (uintptr_t)from | (uintptr_t)bytes) & 15) {  // scales of few heads
    for (long long i = ((long long)part * kThreads + threadIdx.x) * 4; i < bytes; i += (long long)parts * kThreads * 4)
      *reinterpret_cast<uint32_t *>(to + i) = *reinterpret_cast<const uint32_t *>(from + i);
    return;
  }
  const long long step = (long long)parts * kThreads * 16;
  long long i = ((long long)part * kThreads + threadIdx.x) * 16;
  for (; i + 3 * step < bytes; i += 4 * step) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; k++) x[k] = *reinterpret_cast<const uint4 *>(from + i + k * step);
#pragma unroll
    for (int k = 0; k < 4; k++) *reinterpret_cast<uint4 *>(to + i + k * step) = x[k];
  }
  for (; i < bytes; i += step) *reinterpret_cast<uint4 *>(to + i) = *reinterpret_cast<const uint4 *>(from + i);
}

__global__ void __launch_bounds__(kThreads) gdn_kv_copy_kernel(const CopyPagesArgs a, const int parts) {
  __shared__ int own_src[kOwn], own_dst[kOwn], bad[kOwn];
  const int tid = threadIdx.x, part = blockIdx.x % parts;
  const int step = gridDim.x / parts;  // pairs of all blocks at a time
  for (long long i0 = blockIdx.x / parts; i0 < a.n; i0 += (long long)step * kOwn) {
    __syncthreads();
    const int mine = (int)min((long long)kOwn, (a.n - i0 + step - 1) / step);
    if (tid < mine) {
      const int i = (int)(i0 + (long long)tid * step);
      own_src[tid] = __ldg(a.src + i);
      own_dst[tid] = __ldg(a.dst + i);
      bad[tid] = (unsigned)own_src[tid] >= (unsigned)a.n_pages || (unsigned)own_dst[tid] >= (unsigned)a.n_pages;
    }
    __syncthreads();
    for (int j = tid; j < a.n; j += kThreads) {
      const int s = __ldg(a.src + j), d = __ldg(a.dst + j);
      for (int k = 0; k < mine; k++)
        if ((s == own_dst[k] || d == own_dst[k]) && j != i0 + (long long)k * step) bad[k] = 1;
    }
    __syncthreads();
    for (int k = 0; k < mine; k++) {
      if (bad[k]) {
        if (tid == 0 && a.flags) atomicOr(a.flags, kFlagBadSeqlens);
        continue;
      }
      if (own_src[k] == own_dst[k]) continue;  // nothing to do
#pragma unroll
      for (int x = 0; x < 4; x++)
        if (a.base[x]) copy(a.base[x] + own_dst[k] * a.bytes[x], a.base[x] + own_src[k] * a.bytes[x], a.bytes[x], part, parts);
    }
  }
}

}  // namespace

cudaError_t launch_kv_copy_pages(const CopyPagesArgs &a, cudaStream_t stream) {
  const long long most = 4LL * sm_count();  // blocks that the GPU holds
  const long long pairs = a.n < most ? a.n : most;
  const long long pieces = (a.bytes[0] + kThreads * 16 - 1) / (kThreads * 16);
  long long parts = most / pairs;
  if (parts > pieces) parts = pieces;
  if (parts < 1) parts = 1;
  gdn_kv_copy_kernel<<<(unsigned)(pairs * parts), kThreads, 0, stream>>>(a, (int)parts);
  return cudaGetLastError();
}

}  // namespace gdn
