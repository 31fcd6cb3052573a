// Expert layer: assignments sorted by expert, the tokens' rows carried to
// their experts and back with weights applied, and the gradients of both.
// The operations are specified in include/tbe_experts.h.
#include <type_traits>

#include "internal.h"
#include "rows.cuh"
#include "sort.cuh"
#include "tbe_experts.h"

namespace tbe {
namespace {

// ---------------------------------------------------------------------- sort
//
// A counting sort: a warp takes a contiguous chunk of the assignments and counts
// its experts in its own row of shared memory; the rows are scanned over (expert,
// CTA, warp); then each warp walks its chunk again, 32 assignments at a time,
// giving each its place: the warp's running count of the expert plus the number
// of lower lanes with the same expert.  Stable by construction, no atomics on
// results.  Dropped assignments are counted as expert E, which comes last.
//
// Up to kSortOneLaunch assignments it is one launch of one cluster, whose CTAs read
// one another's totals in shared memory; above, three launches over the whole GPU
// (count, scan, rank), whose totals stand in the part of `position` that their
// CTA writes last.  Both measured (64 experts): 65536 assignments 9.0 us in one
// launch and 11.8 in three, 131072 13.3 and 13.2, 262144 21.7 and 12.6, a million 70
// and 25 us.
constexpr int kSortUnroll = 4;      // rounds of 32 assignments whose loads are in flight
constexpr int kSortPerCta = 2048;   // assignments from which another CTA pays
constexpr int kSortOneLaunch = 131072;
constexpr int kSortGridChunk = 4096;  // assignments of a CTA of three launches, at least
constexpr int kSortGridCtas = 304;
constexpr int kScanCtas = 8;
static_assert(kSortGridChunk > TBE_MAX_EXPERTS, "a CTA's totals fit its part of position");

template <typename IdT>
__device__ __forceinline__ int expert_of(IdT e, int experts) {
  return e >= 0 && e < static_cast<IdT>(experts) ? static_cast<int>(e) : experts;
}

// Every warp's counts of its chunk, count[warp][expert], and their sums over
// the warps, total[expert].  The whole CTA; ends before a barrier.
template <typename IdT>
__device__ __forceinline__ void count_chunks(const IdT* ids, Chunk c, int experts, int* count,
                                             int* total) {
  const int buckets = experts + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * buckets; i += blockDim.x) count[i] = 0;
  __syncthreads();
  int* mine = count + warp * buckets;
  for (int64_t a0 = c.first + lane; a0 < c.last; a0 += 32 * kSortUnroll) {
    IdT e[kSortUnroll];
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) e[u] = a0 + 32 * u < c.last ? ids[a0 + 32 * u] : IdT(0);
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u)
      if (a0 + 32 * u < c.last) atomicAdd(mine + expert_of(e[u], experts), 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < buckets; e += blockDim.x) {
    int sum = 0;
#pragma unroll 16
    for (int w = 0; w < kSortWarps; ++w) sum += count[w * buckets + e];
    total[e] = sum;
  }
}

template <typename IdT>
__device__ __forceinline__ void rank_chunk(const IdT* ids, Chunk c, int experts, int* mine,
                                           int* source, int* position) {
  const int lane = threadIdx.x & 31;
  for (int64_t a0 = c.first; a0 < c.last; a0 += 32 * kSortUnroll) {
    IdT id[kSortUnroll];
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      const int64_t a = a0 + 32 * u + lane;
      id[u] = a < c.last ? ids[a] : IdT(0);
    }
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      const int64_t a = a0 + 32 * u + lane;
      const bool on = a < c.last;
      const int e = on ? expert_of(id[u], experts) : -1;
      const unsigned same = __match_any_sync(kAll, e);
      int place = 0;
      if (on) place = mine[e] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (on && (same >> lane) == 1u) mine[e] = place + 1;  // the highest lane of its expert
      __syncwarp();
      if (on) {
        position[a] = e < experts ? place : -1;
        source[place] = e < experts ? static_cast<int>(a) : -1;
      }
    }
  }
}

template <typename IdT>
__global__ void __launch_bounds__(kSortWarps * 32)
    expert_sort_kernel(const IdT* __restrict__ ids, int n, int experts, int* __restrict__ offsets,
                       int* __restrict__ source, int* __restrict__ position) {
  extern __shared__ int sort_smem[];
  __shared__ int warp_sum[kSortWarps];
  const int buckets = experts + 1;
  int* total = sort_smem;            // [buckets] this CTA's assignments of each expert
  int* count = sort_smem + buckets;  // [kSortWarps][buckets]
  const int ctas = gridDim.x, rank = blockIdx.x;  // one cluster
  const int warps = ctas * kSortWarps;
  const int64_t per_warp = (static_cast<int64_t>(n) + warps * 32 - 1) / (warps * 32) * 32;
  const Chunk chunk = warp_chunk(n, rank * kSortWarps * per_warp, per_warp);
  count_chunks(ids, chunk, experts, count, total);
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  int carry = 0;
  for (int e0 = 0; e0 < buckets; e0 += blockDim.x) {  // one expert per thread, in rounds
    const int e = e0 + threadIdx.x;
    int all = 0, before_me = 0;
    if (e < buckets) {
      if (ctas == 1) {
        all = total[e];
      } else {
        int c[kSortMostCtas];
#pragma unroll
        for (int r = 0; r < kSortMostCtas; ++r) c[r] = r < ctas ? load_from_cta(total + e, r) : 0;
#pragma unroll
        for (int r = 0; r < kSortMostCtas; ++r) {
          all += c[r];
          before_me += r < rank ? c[r] : 0;
        }
      }
    }
    int sum;
    const int at = carry + block_scan(all, warp_sum, &sum);
    carry += sum;
    if (e < buckets) {
      if (rank == 0) offsets[e] = at;  // offsets[E]: the first dropped place, the number kept
      counts_to_places(count, buckets, e, at + before_me);
    }
  }
  __syncthreads();
  if (ctas > 1) cluster_arrive();  // this CTA reads no other's memory any more
  rank_chunk(ids, chunk, experts, count + (threadIdx.x >> 5) * buckets, source, position);
  if (ctas > 1) cluster_wait();  // no CTA ends while another may read its totals
}

// The three launches.  The CTAs have equal parts of the assignments (the first n % ctas one
// more), and a CTA's totals, then its first places, stand at the start of its part of position
// until it ranks them.
template <typename IdT>
__global__ void __launch_bounds__(kSortWarps * 32)
    expert_count_kernel(const IdT* __restrict__ ids, int n, int experts,
                        int* __restrict__ position) {
  extern __shared__ int sort_smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int buckets = experts + 1;
  count_chunks(ids, my_chunk(n), experts, sort_smem + buckets, sort_smem);
  int* row = position + cta_first(n, blockIdx.x, gridDim.x);
  for (int e = threadIdx.x; e < buckets; e += blockDim.x)  // the entries it summed: no barrier
    row[e] = sort_smem[e];
}

// One CTA, or for many experts a cluster whose CTAs have equal shares of them; `segments`
// threads an expert, each over a run of the counting CTAs.
__global__ void __launch_bounds__(kSortWarps * 32)
    expert_scan_kernel(int n, int experts, int ctas, int share, int segments,
                       int* __restrict__ offsets, int* __restrict__ position) {
  __shared__ int warp_sum[kSortWarps];
  __shared__ int total;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int run = (ctas + segments - 1) / segments;
  // an expert's threads are neighbours, so the scan runs over (expert, run of CTAs)
  const int in_share = static_cast<int>(threadIdx.x) / segments;
  const int e = static_cast<int>(blockIdx.x) * share + in_share;
  const bool on = in_share < share && e <= experts;
  const int c0 = static_cast<int>(threadIdx.x) % segments * run;
  const int c1 = on ? (c0 + run < ctas ? c0 + run : ctas) : c0;
  int sum = 0;
#pragma unroll 8
  for (int c = c0; c < c1; ++c) sum += position[cta_first(n, c, ctas) + e];
  int all;
  int at = block_scan(sum, warp_sum, &all);
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) total = all;
    cluster_arrive();
    cluster_wait();
    int before[kScanCtas];
#pragma unroll
    for (int r = 0; r < kScanCtas; ++r)
      before[r] = r < static_cast<int>(blockIdx.x) ? load_from_cta(&total, r) : 0;
#pragma unroll
    for (int r = 0; r < kScanCtas; ++r) at += before[r];
    cluster_arrive();
  }
  if (on && c0 == 0) offsets[e] = at;
#pragma unroll 8
  for (int c = c0; c < c1; ++c) {
    int* p = position + cta_first(n, c, ctas) + e;
    const int v = *p;
    *p = at;
    at += v;
  }
  if (gridDim.x > 1) cluster_wait();  // no CTA ends while another may read its total
}

template <typename IdT>
__global__ void __launch_bounds__(kSortWarps * 32)
    expert_rank_kernel(const IdT* __restrict__ ids, int n, int experts,
                       int* __restrict__ source, int* position) {
  extern __shared__ int sort_smem[];
  const int buckets = experts + 1;
  int* count = sort_smem + buckets;
  const Chunk chunk = my_chunk(n);
  count_chunks(ids, chunk, experts, count, sort_smem);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int* row = position + cta_first(n, blockIdx.x, gridDim.x);
  for (int e = threadIdx.x; e < buckets; e += blockDim.x)
    counts_to_places(count, buckets, e, row[e]);
  __syncthreads();  // the places have been read: position may be written
  rank_chunk(ids, chunk, experts, count + (threadIdx.x >> 5) * buckets, source, position);
}

// --------------------------------------------------------------- moving rows
//
// Memory bounds these kernels: a token's row is read once and its k rows are
// written, or the k rows are read and one is written.  A group of threads
// serves one token, `log_group` threads each; the block's 256 threads serve
// several narrow tokens or one wide one.  Rows that do not begin on 16-byte
// boundaries are moved in 16-byte vectors all the same (inner_span, load_vec).
// 65536 tokens x 2048 bf16, four experts each: dispatch 202 us (6.6 TB/s), combine 197
// (6.8), its gradient 356 (6.8); 4097 x 1001 fp16, three each: 10.4, 12.6 and 13.0 us.
constexpr int kMoveThreads = 256;

struct Group {
  int64_t token;
  int t, size;
};

__device__ __forceinline__ Group my_group(int log_group) {
  const int size = 1 << log_group;
  return {static_cast<int64_t>(blockIdx.x) * (kMoveThreads >> log_group) +
              (threadIdx.x >> log_group),
          static_cast<int>(threadIdx.x & (size - 1)), size};
}

__device__ __forceinline__ int64_t kept_rows(const int* offsets, int experts, int64_t rows) {
  const int64_t m = offsets[experts];
  return m < 0 ? 0 : m > rows ? rows : m;
}

// Clears rows [first, last): those of dropped assignments.
template <typename T, bool kAligned>
__device__ __forceinline__ void clear_rows(int t, int threads, int width, int64_t first,
                                           int64_t last, T* rows, int64_t stride) {
  Pack<T, kVec<T>> zero;
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) zero.v[i] = from_f32<T>(0.f);
  for (int64_t r = first; r < last; ++r) {
    T* row = rows + r * stride;
    const Span s = inner_span<T, kAligned>(row, width);
    for (int e = s.lo + t * kVec<T>; e < s.hi; e += threads * kVec<T>) store_vec(row + e, zero);
    for_ends(s, width, t, threads, [&](int e) { row[e] = from_f32<T>(0.f); });
  }
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kMoveThreads)
    dispatch_kernel(const T* __restrict__ x, int64_t tokens, int k, int width, int64_t x_stride,
                    const int* __restrict__ offsets, int experts, const int* __restrict__ position,
                    T* __restrict__ rows, int64_t rows_stride, int log_group) {
  const Group g = my_group(log_group);
  if (g.token >= tokens) return;
  const int64_t all = tokens * k;
  const int* pos = position + g.token * k;
  const T* src = x + g.token * x_stride;
  const int step = g.size * kVec<T>;
  if constexpr (kAligned) {
    for (int e = g.t * kVec<T>; e < width; e += 2 * step) {
      const bool two = e + step < width;
      const Pack<T, kVec<T>> v0 = load_vec<T, true>(src + e);
      Pack<T, kVec<T>> v1 = v0;
      if (two) v1 = load_vec<T, true>(src + e + step);
      for (int j = 0; j < k; ++j) {
        const int64_t p = pos[j];
        if (p < 0 || p >= all) continue;
        T* row = rows + p * rows_stride;
        store_vec(row + e, v0);
        if (two) store_vec(row + e + step, v1);
      }
    }
  } else {
    for (int j = 0; j < k; ++j) {  // every row has boundaries of its own
      const int64_t p = pos[j];
      if (p < 0 || p >= all) continue;
      T* row = rows + p * rows_stride;
      const Span s = inner_span<T, false>(row, width);
      for (int e = s.lo + g.t * kVec<T>; e < s.hi; e += step)
        store_vec(row + e, load_vec<T, false>(src + e));
      for_ends(s, width, g.t, g.size, [&](int e) { row[e] = src[e]; });
    }
  }
  const int64_t kept = kept_rows(offsets, experts, all), mine = g.token * k;
  clear_rows<T, kAligned>(g.t, g.size, width, mine < kept ? kept : mine, mine + k, rows,
                          rows_stride);
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kMoveThreads, sizeof(T) == 4 ? 6 : 5)
    combine_kernel(const T* __restrict__ y, int64_t tokens, int k, int width, int64_t y_stride,
                   const int* __restrict__ position, const float* __restrict__ weights,
                   T* __restrict__ out, int64_t out_stride, int log_group) {
  constexpr int kRows = 4;  // rows whose loads are in flight
  const Group g = my_group(log_group);
  if (g.token >= tokens) return;
  const int64_t all = tokens * k;
  const int* pos = position + g.token * k;
  const float* w = weights + g.token * k;
  T* dst = out + g.token * out_stride;
  const Span s = inner_span<T, kAligned>(dst, width);
  for (int e = s.lo + g.t * kVec<T>; e < s.hi; e += g.size * kVec<T>) {
    float acc[kVec<T>];
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += kRows) {
      Pack<T, kVec<T>> v[kRows];
      float f[kRows];
      bool on[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t p = j0 + u < k ? pos[j0 + u] : -1;
        on[u] = p >= 0 && p < all;
        if (on[u]) {
          f[u] = weights ? w[j0 + u] : 1.f;
          v[u] = load_vec<T, kAligned>(y + p * y_stride + e);
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (on[u]) {
          float r[kVec<T>];
          to_floats<T>(v[u], r);
#pragma unroll
          for (int i = 0; i < kVec<T>; ++i) acc[i] = fmaf(f[u], r[i], acc[i]);
        }
    }
    store_vec(dst + e, from_floats<T>(acc));
  }
  if constexpr (!kAligned)
    for_ends(s, width, g.t, g.size, [&](int e) {
      float acc = 0.f;
      for (int j = 0; j < k; ++j) {
        const int64_t p = pos[j];
        if (p >= 0 && p < all) acc = fmaf(weights ? w[j] : 1.f, to_f32(y[p * y_stride + e]), acc);
      }
      dst[e] = from_f32<T>(acc);
    });
}

// Sum over a group of `size` lanes; the whole warp calls it.
__device__ __forceinline__ float group_sum(float v, int size) {
  for (int o = size >> 1; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The gradients of combine, a group (a warp, or a part of one for narrow rows) a token:
// grad_out's row is read once for four of the token's rows, whose loads are in flight together
// (65536 tokens x 4 rows of 2048 bf16: 356 us, a row after the other 405).
template <typename T>
__global__ void __launch_bounds__(kMoveThreads, 4)
    combine_backward_by_token(const T* __restrict__ grad_out, const T* __restrict__ y,
                              int64_t tokens, int k, int width, int64_t go_stride,
                              int64_t y_stride, const int* __restrict__ offsets, int experts,
                              const int* __restrict__ position,
                              const float* __restrict__ weights, T* __restrict__ grad_y,
                              int64_t gy_stride, float* __restrict__ grad_weights,
                              int log_group) {
  constexpr int kRows = 4;
  const Group g = my_group(log_group);
  const bool live = g.token < tokens;  // the others take part in the sums
  const int64_t all = tokens * k, mine = g.token * k;
  const T* go = grad_out + g.token * go_stride;
  for (int j0 = 0; j0 < k; j0 += kRows) {
    int64_t p[kRows];
    float f[kRows], dot[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      p[u] = live && j0 + u < k ? position[mine + j0 + u] : -1;
      if (p[u] >= all) p[u] = -1;
      f[u] = p[u] >= 0 && weights ? weights[mine + j0 + u] : 1.f;
      dot[u] = 0.f;
    }
    for (int e = g.t * kVec<T>; live && e < width; e += g.size * kVec<T>) {
      const Pack<T, kVec<T>> gv = load_vec<T, true>(go + e);
      Pack<T, kVec<T>> v[kRows];
      if (grad_weights) {
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (p[u] >= 0) v[u] = load_vec<T, true>(y + p[u] * y_stride + e);
      }
      float d[kVec<T>];
      to_floats<T>(gv, d);
      if (grad_weights) {
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (p[u] >= 0) {
            float r[kVec<T>];
            to_floats<T>(v[u], r);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) dot[u] = fmaf(d[i], r[i], dot[u]);
          }
      }
      if (grad_y) {
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (p[u] >= 0) {
            float r[kVec<T>];
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) r[i] = f[u] * d[i];
            store_vec(grad_y + p[u] * gy_stride + e, from_floats<T>(r));
          }
      }
    }
    if (grad_weights) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const float sum = group_sum(dot[u], g.size);
        if (live && g.t == 0 && j0 + u < k) grad_weights[mine + j0 + u] = sum;
      }
    }
  }
  if (!grad_y || !live) return;
  const int64_t kept = kept_rows(offsets, experts, all);
  clear_rows<T, true>(g.t, g.size, width, mine < kept ? kept : mine, mine + k, grad_y, gy_stride);
}

// The same, a group an assignment: for rows that share no boundaries, and for tokens
// too few to fill the GPU.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kMoveThreads)
    combine_backward_by_assignment(const T* __restrict__ grad_out, const T* __restrict__ y,
                                   int64_t tokens, int k, int width, int64_t go_stride,
                                   int64_t y_stride, const int* __restrict__ offsets, int experts,
                                   const int* __restrict__ position,
                                   const float* __restrict__ weights, T* __restrict__ grad_y,
                                   int64_t gy_stride, float* __restrict__ grad_weights,
                                   int log_group) {
  const Group g = my_group(log_group);
  const int64_t a = g.token, all = tokens * k;  // a group is an assignment here
  const bool live = a < all;  // the others take part in the sums
  const int64_t p = live ? position[a] : -1;
  const bool on = p >= 0 && p < all;
  float dot = 0.f;
  if (on) {
    const float f = weights ? weights[a] : 1.f;
    const T* go = grad_out + a / k * go_stride;
    const T* yr = y + p * y_stride;
    T* gy = grad_y + p * gy_stride;
    const Span s = inner_span<T, kAligned>(grad_y ? gy : yr, width);
#pragma unroll 2
    for (int e = s.lo + g.t * kVec<T>; e < s.hi; e += g.size * kVec<T>) {
      const Pack<T, kVec<T>> gv = load_vec<T, kAligned, true>(go + e);
      float d[kVec<T>], r[kVec<T>];
      if (grad_weights) {
        const Pack<T, kVec<T>> yv = load_vec<T, kAligned, true>(yr + e);
        to_floats<T>(gv, d);
        to_floats<T>(yv, r);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) dot = fmaf(d[i], r[i], dot);
      } else {
        to_floats<T>(gv, d);
      }
      if (grad_y) {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) r[i] = f * d[i];
        store_vec(gy + e, from_floats<T>(r));
      }
    }
    if constexpr (!kAligned)
      for_ends(s, width, g.t, g.size, [&](int e) {
        const float d = to_f32(go[e]);
        if (grad_weights) dot = fmaf(d, to_f32(yr[e]), dot);
        if (grad_y) gy[e] = from_f32<T>(f * d);
      });
  }
  if (grad_weights) {
    dot = group_sum(dot, g.size);
    if (live && g.t == 0) grad_weights[a] = dot;
  }
  if (grad_y && live && a >= kept_rows(offsets, experts, all))
    clear_rows<T, kAligned>(g.t, g.size, width, a, a + 1, grad_y, gy_stride);
}

// -------------------------------------------------------------- host checks

tbe_status check_rows(int32_t dtype, int64_t tokens, int32_t k, int64_t width) {
  if (tokens < 0 || k < 1 || width < 0) return TBE_EINVAL;
  if (!dtype_bytes(dtype)) return TBE_EUNSUPPORTED;
  if (tokens > INT32_MAX / k || width > INT32_MAX / 2) return TBE_EUNSUPPORTED;
  return TBE_OK;
}

bool check_matrix(const void* p, int32_t dtype, int64_t stride, int64_t width) {
  return p && stride >= width && aligned_to(p, dtype_bytes(dtype));
}

Bytes bytes_of(const void* p, int32_t dtype, int64_t rows, int64_t width, int64_t stride) {
  const int64_t b = dtype_bytes(dtype);
  return {p, rows, width * b, stride * b};
}

bool check_plan(const int32_t* offsets, const int32_t* position) {
  return offsets && position && aligned_to(offsets, 4) && aligned_to(position, 4);
}

// Whether rows starting at p, `stride` elements apart, can be moved in
// 16-byte vectors from end to end.
bool vector_rows(const void* p, int bytes, int64_t stride, int64_t width) {
  return aligned_to(p, 16) && stride * bytes % 16 == 0 && width * bytes % 16 == 0;
}

// Threads of a group: one for each 16-byte place of a row of `width` elements
// (and one more where rows do not begin on boundaries) while the tokens are few
// and latency counts; a quarter of that, at least a warp, once they fill the GPU,
// so that a thread has several loads in flight.
int log_group_of(int64_t tokens, int64_t width, int bytes, bool aligned) {
  int64_t places = (width * bytes + 15) / 16 + (aligned ? 0 : 1);
  if (tokens * places > 152 * 2048 && places > 128) places = (places + 3) / 4;
  int lg = 0;
  while (lg < 8 && (1 << lg) < places) ++lg;
  return lg;
}

int64_t group_blocks(int64_t tokens, int log_group) {
  const int per = kMoveThreads >> log_group;
  return (tokens + per - 1) / per;
}

tbe_status launched() {
  note_launch();
  return cudaGetLastError() == cudaSuccess ? TBE_OK : TBE_ECUDA;
}

// Calls f with a value of the row type and whether rows are aligned, as a constant.
template <typename F>
tbe_status for_dtype(int32_t dtype, bool aligned, F f) {
  using Yes = std::true_type;
  using No = std::false_type;
  if (dtype == TBE_DT_F32) return aligned ? f(float{}, Yes{}) : f(float{}, No{});
  if (dtype == TBE_DT_F16) return aligned ? f(__half{}, Yes{}) : f(__half{}, No{});
  return aligned ? f(__nv_bfloat16{}, Yes{}) : f(__nv_bfloat16{}, No{});
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_expert_sort(const void* ids, int32_t index_dtype, int64_t tokens,
                                      int32_t k, int32_t experts, int32_t* offsets,
                                      int32_t* source, int32_t* position, void* stream) {
  if (tokens < 0 || k < 1 || experts < 1 || !offsets) return TBE_EINVAL;
  if (tokens && (!ids || !source || !position)) return TBE_EINVAL;
  if (index_dtype != TBE_DT_I32 && index_dtype != TBE_DT_I64) return TBE_EUNSUPPORTED;
  if (tokens > INT32_MAX / k || experts > TBE_MAX_EXPERTS) return TBE_EUNSUPPORTED;
  if (!aligned_to(ids, index_dtype == TBE_DT_I32 ? 4 : 8) || !aligned_to(offsets, 4) ||
      !aligned_to(source, 4) || !aligned_to(position, 4))
    return TBE_EINVAL;
  const int n = static_cast<int>(tokens * k);
  const Bytes in_out[4] = {run_of(ids, int64_t(n) * (index_dtype == TBE_DT_I32 ? 4 : 8)),
                           run_of(offsets, (int64_t(experts) + 1) * 4),
                           run_of(source, int64_t(n) * 4), run_of(position, int64_t(n) * 4)};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(in_out[i], in_out[j])) return TBE_EINVAL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = static_cast<size_t>(kSortWarps + 1) * (experts + 1) * 4;
  // shared memory above 48 KB and clusters above eight CTAs have to be asked for
  const auto room_for = [&](auto kernel) {
    return smem <= 48 * 1024 ||
           cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (kSortWarps + 1) * (TBE_MAX_EXPERTS + 1) * 4) == cudaSuccess;
  };
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kSortWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  const auto one_launch = [&](auto* p) {
    using IdT = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    const auto kernel = expert_sort_kernel<IdT>;
    int ctas = 1;
    while (ctas < kSortMostCtas && n > ctas * kSortPerCta) ctas *= 2;
    if (!room_for(kernel) ||
        (ctas > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                          1) != cudaSuccess))
      return refused();
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, p, n, experts, offsets, source, position) != cudaSuccess)
      return refused();
    return launched();
  };
  const auto three_launches = [&](auto* p) {
    using IdT = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    const int ctas = n / kSortGridChunk < kSortGridCtas ? n / kSortGridChunk : kSortGridCtas;
    const auto count = expert_count_kernel<IdT>;
    const auto rank = expert_rank_kernel<IdT>;
    if (!room_for(count) || !room_for(rank)) return refused();
    const int scan_ctas = experts < 256 ? 1 : kScanCtas;
    const int share = (experts + scan_ctas) / scan_ctas;  // of the E + 1 buckets
    int segments = 1;
    while (segments * 2 * share <= kSortWarps * 32) segments *= 2;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.numAttrs = 0;
    if (cudaLaunchKernelEx(&cfg, count, p, n, experts, position) != cudaSuccess)
      return refused();
    note_launch();
    // the next two begin while the launch before them ends (griddepcontrol.wait)
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(scan_ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(static_cast<unsigned>(scan_ctas));
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, expert_scan_kernel, n, experts, ctas, share, segments, offsets,
                           position) != cudaSuccess)
      return refused();
    cfg.numAttrs = 1;
    note_launch();
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.dynamicSmemBytes = smem;
    if (cudaLaunchKernelEx(&cfg, rank, p, n, experts, source, position) != cudaSuccess)
      return refused();
    return launched();
  };
  const auto go = [&](auto* p) { return n <= kSortOneLaunch ? one_launch(p) : three_launches(p); };
  return index_dtype == TBE_DT_I32 ? go(static_cast<const int32_t*>(ids))
                                   : go(static_cast<const int64_t*>(ids));
}

extern "C" tbe_status tbe_expert_dispatch(const void* x, int32_t dtype, int64_t tokens, int32_t k,
                                          int64_t width, int64_t x_stride, const int32_t* offsets,
                                          int32_t experts, const int32_t* position, void* rows,
                                          int64_t rows_stride, void* stream) {
  const tbe_status bad = check_rows(dtype, tokens, k, width);
  if (bad != TBE_OK) return bad;
  if (!tokens || !width) return TBE_OK;
  if (experts < 1 || !check_plan(offsets, position) || !check_matrix(x, dtype, x_stride, width) ||
      !check_matrix(rows, dtype, rows_stride, width) ||
      overlap(bytes_of(x, dtype, tokens, width, x_stride),
              bytes_of(rows, dtype, tokens * k, width, rows_stride)))
    return TBE_EINVAL;
  int b = dtype_bytes(dtype);
  const bool vec = vector_rows(x, b, x_stride, width) && vector_rows(rows, b, rows_stride, width);
  // Rows are carried as they are, so 16-bit rows on 4-byte boundaries go as 4-byte elements: half
  // as many at the rows' ends (93576 x 20 fp16, eight experts each: 16.8 us instead of 29.2).
  if (!vec && b == 2 && width % 2 == 0 && x_stride % 2 == 0 && rows_stride % 2 == 0 &&
      aligned_to(x, 4) && aligned_to(rows, 4)) {
    dtype = TBE_DT_F32;
    b = 4;
    width /= 2;
    x_stride /= 2;
    rows_stride /= 2;
  }
  return for_dtype(dtype, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr bool kAligned = decltype(v)::value;
    const int lg = log_group_of(tokens, width, b, kAligned);
    dispatch_kernel<T, kAligned><<<static_cast<unsigned>(group_blocks(tokens, lg)), kMoveThreads, 0,
                            static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(x), tokens, k, static_cast<int>(width), x_stride, offsets, experts,
        position, static_cast<T*>(rows), rows_stride, lg);
    return launched();
  });
}

extern "C" tbe_status tbe_expert_combine(const void* y, int32_t dtype, int64_t tokens, int32_t k,
                                         int64_t width, int64_t y_stride, const int32_t* position,
                                         const float* weights, void* out, int64_t out_stride,
                                         void* stream) {
  const tbe_status bad = check_rows(dtype, tokens, k, width);
  if (bad != TBE_OK) return bad;
  if (!tokens || !width) return TBE_OK;
  if (!check_plan(position, position) || !check_matrix(y, dtype, y_stride, width) ||
      !check_matrix(out, dtype, out_stride, width) || !aligned_to(weights, 4) ||
      overlap(bytes_of(y, dtype, tokens * k, width, y_stride),
              bytes_of(out, dtype, tokens, width, out_stride)))
    return TBE_EINVAL;
  const int b = dtype_bytes(dtype);
  const bool vec = vector_rows(y, b, y_stride, width) && vector_rows(out, b, out_stride, width);
  return for_dtype(dtype, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr bool kAligned = decltype(v)::value;
    const int lg = log_group_of(tokens, width, b, kAligned);
    combine_kernel<T, kAligned><<<static_cast<unsigned>(group_blocks(tokens, lg)), kMoveThreads, 0,
                           static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(y), tokens, k, static_cast<int>(width), y_stride, position, weights,
        static_cast<T*>(out), out_stride, lg);
    return launched();
  });
}

extern "C" tbe_status tbe_expert_combine_backward(
    const void* grad_out, const void* y, int32_t dtype, int64_t tokens, int32_t k, int64_t width,
    int64_t grad_out_stride, int64_t y_stride, const int32_t* offsets, int32_t experts,
    const int32_t* position, const float* weights, void* grad_y, int64_t grad_y_stride,
    float* grad_weights, void* stream) {
  const tbe_status bad = check_rows(dtype, tokens, k, width);
  if (bad != TBE_OK) return bad;
  if (!tokens || (!grad_y && !grad_weights)) return TBE_OK;
  if (experts < 1 || !check_plan(offsets, position) || !aligned_to(weights, 4) ||
      !aligned_to(grad_weights, 4))
    return TBE_EINVAL;
  if (width && (!check_matrix(grad_out, dtype, grad_out_stride, width) ||
                (grad_weights && !check_matrix(y, dtype, y_stride, width)) ||
                (grad_y && !check_matrix(grad_y, dtype, grad_y_stride, width))))
    return TBE_EINVAL;
  const Bytes gy = bytes_of(grad_y, dtype, tokens * k, width, grad_y_stride);
  if (overlap(bytes_of(grad_out, dtype, tokens, width, grad_out_stride), gy) ||
      (grad_weights && overlap(bytes_of(y, dtype, tokens * k, width, y_stride), gy)))
    return TBE_EINVAL;
  const int b = dtype_bytes(dtype);
  const bool vec = vector_rows(grad_out, b, grad_out_stride, width) &&
                   (!grad_weights || vector_rows(y, b, y_stride, width)) &&
                   (!grad_y || vector_rows(grad_y, b, grad_y_stride, width));
  return for_dtype(dtype, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr bool kAligned = decltype(v)::value;
    // a group a token, if that fills the GPU (24 warps a multiprocessor)
    const bool by_token = kAligned && tokens * ((width * b + 511) / 512) >= 152 * 24;
    const auto kernel = by_token ? combine_backward_by_token<T>
                                 : combine_backward_by_assignment<T, kAligned>;
    const int64_t groups = by_token ? tokens : tokens * k;
    int lg = log_group_of(groups, width, b, kAligned);
    if (lg > 5) lg = 5;
    kernel<<<static_cast<unsigned>(group_blocks(groups, lg)), kMoveThreads, 0,
             static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(grad_out), static_cast<const T*>(y), tokens, k,
        static_cast<int>(width), grad_out_stride, y_stride, offsets, experts, position, weights,
        static_cast<T*>(grad_y), grad_y_stride, grad_weights, lg);
    return launched();
  });
}
