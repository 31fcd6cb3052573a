// What the counting sorts share: the split of a CTA's entries over its warps, the
// scans, and clusters whose CTAs read one another's totals.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace tbe {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSortWarps = 32;
constexpr int kSortMostCtas = 16;

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ int load_from_cta(const int* p, int rank) {
  const unsigned addr = static_cast<unsigned>(__cvta_generic_to_shared(p));
  unsigned remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// Entries [first, last) of a warp.
struct Chunk {
  int64_t first, last;
};
__device__ __forceinline__ Chunk warp_chunk(int64_t n, int64_t cta_first, int64_t per_warp) {
  const int64_t first = cta_first + (threadIdx.x >> 5) * per_warp;
  return {first, first + per_warp < n ? first + per_warp : n};
}

// Turns bucket e's counts into every warp's first place, from `at` on.
__device__ __forceinline__ void counts_to_places(int* count, int buckets, int e, int at) {
#pragma unroll 16
  for (int w = 0; w < kSortWarps; ++w) {
    const int c = count[w * buckets + e];
    count[w * buckets + e] = at;
    at += c;
  }
}

// Exclusive scan over the CTA's threads, and the sum; kSortWarps warps.
__device__ __forceinline__ int block_scan(int v, int* warp_sum, int* sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int sums = warp_sum[lane];  // scanned by every warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, sums, o);
    if (lane >= o) sums += y;
  }
  const int before = warp ? __shfl_sync(kAll, sums, warp - 1) : 0;
  *sum = __shfl_sync(kAll, sums, 31);
  __syncthreads();
  return before + incl - v;
}

// Equal parts of n entries for `ctas` CTAs (the first n % ctas have one more).
__device__ __forceinline__ int64_t cta_first(int n, int c, int ctas) {
  const int rest = n % ctas;
  return static_cast<int64_t>(n / ctas) * c + (c < rest ? c : rest);
}
__device__ __forceinline__ Chunk my_chunk(int n) {
  const int64_t first = cta_first(n, blockIdx.x, gridDim.x);
  const int64_t last = cta_first(n, blockIdx.x + 1, gridDim.x);
  const int64_t per_warp = (last - first + kSortWarps * 32 - 1) / (kSortWarps * 32) * 32;
  return warp_chunk(last, first, per_warp);
}

}  // namespace tbe
