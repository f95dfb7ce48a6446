// gdn_kv_copy.cu -- copies whole pages of a cache: page src[i] to page dst[i], keys,
// values and, of a cache in 8 bits, scales, as when a sequence forks (its last page,
// which both go on writing) or a pool is put in order.
//
// Every pair reads what was there before the call: a page that is the destination of
// two pairs, or of one and the source of another, is left as it is, and reported.  A
// block looks that up for the pairs that it copies, kOwn at a time, in chains by their
// destinations, while it goes through all pairs once.  So it takes n^2 / kOwn reads in
// all: 1.7 ms for 131072 pairs, 66 for 2^20, the most of a call, whatever order their pages
// have (32 pairs compared one by one, without chains: 11 and 649; chains by the last bits
// of a page's number, destinations in order: 8.4 and 507).
//
// A copy, bound by memory: 16 bytes to a thread, eight in flight (with four, in blocks of
// 512 threads, 4096 pages of an 8-bit cache took 6 us more); a pair is split between
// blocks while there are fewer pairs than the SMs want.  These 4096 pages: 171 us, 6.3
// TB/s read and written; 32 pages of 64 tokens, 8 heads of 128 in bf16: 4.6 us.
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kFlight = 8;
constexpr int kPiece = 8192;  // bytes of an array's page for a block, at least
constexpr int kOwn = 128;
constexpr int kHeads = 256;

// The chain that a page is in.  Pages in order or evenly spaced, as where a pool is put in
// order, are spread like random ones: a block's own pairs are thousands apart in the list, so by their
// last bits alone its destinations fell into four chains, or one.
__host__ __device__ __forceinline__ unsigned chain_of(int page) {
  uint32_t x = (uint32_t)page * 0x9e3779b1u;
  x = (x ^ x >> 15) * 0x85ebca77u;
  return x >> 24;
}
static_assert(kHeads == 256, "chain_of()");

// A part of a page of two arrays at once, so that a small part's reads are all on their way.
__device__ __forceinline__ void copy(char *const (&base)[2], long long bytes, int dst, int src, int part, int parts) {
  const char *from[2] = {base[0] + src * bytes, base[1] + src * bytes};
  char *to[2] = {base[0] + dst * bytes, base[1] + dst * bytes};
  if (((uintptr_t)to[0] | (uintptr_t)from[0] | (uintptr_t)to[1] | (uintptr_t)from[1] | (uintptr_t)bytes) & 15) {  // scales of few heads
    for (long long i = ((long long)part * kThreads + threadIdx.x) * 4; i < bytes; i += (long long)parts * kThreads * 4)
#pragma unroll
      for (int x = 0; x < 2; x++) *reinterpret_cast<uint32_t *>(to[x] + i) = *reinterpret_cast<const uint32_t *>(from[x] + i);
    return;
  }
  const long long step = (long long)parts * kThreads * 16;
  for (long long i = ((long long)part * kThreads + threadIdx.x) * 16; i < bytes; i += kFlight / 2 * step) {
    uint4 x[2][kFlight / 2];
#pragma unroll
    for (int k = 0; k < kFlight / 2; k++)
      if (i + k * step < bytes) {
        x[0][k] = *reinterpret_cast<const uint4 *>(from[0] + i + k * step);
        x[1][k] = *reinterpret_cast<const uint4 *>(from[1] + i + k * step);
      }
#pragma unroll
    for (int k = 0; k < kFlight / 2; k++)
      if (i + k * step < bytes) {
        *reinterpret_cast<uint4 *>(to[0] + i + k * step) = x[0][k];
        *reinterpret_cast<uint4 *>(to[1] + i + k * step) = x[1][k];
      }
  }
}

__global__ void __launch_bounds__(kThreads) gdn_kv_copy_kernel(const CopyPagesArgs a, const int parts) {
  __shared__ int own_src[kOwn], own_dst[kOwn], bad[kOwn];
  __shared__ int head[kHeads], behind[kOwn];  // own pairs in chains, by their destination
  const int tid = threadIdx.x, part = blockIdx.x % parts;
  const int step = gridDim.x / parts;  // pairs of all blocks at a time
  for (long long i0 = blockIdx.x / parts; i0 < a.n; i0 += (long long)step * kOwn) {
    __syncthreads();
    for (int i = tid; i < kHeads; i += kThreads) head[i] = -1;
    __syncthreads();
    const int mine = (int)min((long long)kOwn, (a.n - i0 + step - 1) / step);
    if (tid < mine) {
      const int i = (int)(i0 + (long long)tid * step);
      own_src[tid] = __ldg(a.src + i);
      own_dst[tid] = __ldg(a.dst + i);
      bad[tid] = (unsigned)own_src[tid] >= (unsigned)a.n_pages || (unsigned)own_dst[tid] >= (unsigned)a.n_pages;
      behind[tid] = atomicExch(&head[chain_of(own_dst[tid])], tid);
    }
    __syncthreads();
#pragma unroll 4
    for (int j = tid; j < a.n; j += kThreads) {
      const int s = __ldg(a.src + j), d = __ldg(a.dst + j);
      auto look = [&](int page) {
        for (int k = head[chain_of(page)]; k >= 0; k = behind[k])
          if (own_dst[k] == page && j != i0 + (long long)k * step) bad[k] = 1;
      };
      look(s);
      look(d);
    }
    __syncthreads();
    for (int k = 0; k < mine; k++) {
      if (bad[k]) {
        if (tid == 0 && a.flags) atomicOr(a.flags, kFlagBadSeqlens);
        continue;
      }
      if (own_src[k] == own_dst[k]) continue;  // nothing to do
      copy({a.base[0], a.base[1]}, a.bytes[0], own_dst[k], own_src[k], part, parts);
      if (a.base[2]) copy({a.base[2], a.base[3]}, a.bytes[2], own_dst[k], own_src[k], part, parts);
    }
  }
}

}  // namespace

cudaError_t launch_kv_copy_pages(const CopyPagesArgs &a, cudaStream_t stream) {
  const long long most = 8LL * sm_count();  // blocks that the GPU holds
  const long long pairs = a.n < most ? a.n : most;
  const long long pieces = (a.bytes[0] + kPiece - 1) / kPiece;
  long long parts = most / pairs;
  if (parts > pieces) parts = pieces;
  if (parts < 1) parts = 1;
  gdn_kv_copy_kernel<<<(unsigned)(pairs * parts), kThreads, 0, stream>>>(a, (int)parts);
  return cudaGetLastError();
}

}  // namespace gdn
