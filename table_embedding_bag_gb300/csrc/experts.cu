// Expert layer: assignments sorted by expert, the tokens' rows carried to
// their experts and back with weights applied, and the gradients of both.
// The operations are specified in include/tbe_experts.h.
#include "internal.h"
#include "rows.cuh"
#include "tbe_experts.h"

namespace tbe {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------------- sort
//
// A counting sort: a warp takes a contiguous chunk of the assignments, counts
// its experts in its own shared-memory row, and after a scan over (expert,
// warp) walks the chunk again, 32 assignments at a time, giving each its place:
// the warp's running count of the expert plus the number of lower lanes with
// the same expert.  Stable by construction, no atomics on results.  Dropped
// assignments are counted as expert E, which comes last.
constexpr int kSortWarps = 32;

template <typename IdT>
__device__ __forceinline__ int expert_of(const IdT* ids, int64_t a, int experts) {
  const IdT e = ids[a];
  return e >= 0 && e < static_cast<IdT>(experts) ? static_cast<int>(e) : experts;
}

template <typename IdT>
__global__ void __launch_bounds__(kSortWarps * 32)
    expert_sort_kernel(const IdT* __restrict__ ids, int n, int experts, int* __restrict__ offsets,
                       int* __restrict__ source, int* __restrict__ position) {
  extern __shared__ int sort_smem[];
  __shared__ int warp_sum[kSortWarps];
  const int buckets = experts + 1;
  int* count = sort_smem;  // [kSortWarps][buckets]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * buckets; i += blockDim.x) count[i] = 0;
  __syncthreads();
  const int64_t chunk = ((static_cast<int64_t>(n) + kSortWarps * 32 - 1) / (kSortWarps * 32)) * 32;
  const int64_t first = warp * chunk;
  const int64_t last = first + chunk < n ? first + chunk : n;
  int* mine = count + warp * buckets;
  for (int64_t a = first + lane; a < last; a += 32) atomicAdd(mine + expert_of(ids, a, experts), 1);
  __syncthreads();
  // exclusive scan over (expert, warp); one expert per thread, in rounds
  int carry = 0;
  for (int e0 = 0; e0 < buckets; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int total = 0;
    if (e < buckets)
      for (int w = 0; w < kSortWarps; ++w) total += count[w * buckets + e];
    int incl = total;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      carry += warp_sum[w];
    }
    int at = before + incl - total;
    if (e < buckets) {
      offsets[e] = at;  // offsets[E]: the first dropped place, the number kept
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = count[w * buckets + e];
        count[w * buckets + e] = at;
        at += c;
      }
    }
    __syncthreads();
  }
  for (int64_t a0 = first; a0 < last; a0 += 32) {
    const int64_t a = a0 + lane;
    const bool on = a < last;
    const unsigned live = __ballot_sync(kAll, on);
    if (on) {
      const int e = expert_of(ids, a, experts);
      const unsigned same = __match_any_sync(live, e);
      const int place = mine[e] + __popc(same & ((1u << lane) - 1));
      __syncwarp(live);
      if ((same >> lane) == 1u) mine[e] = place + 1;  // the highest lane of its expert
      position[a] = e < experts ? place : -1;
      source[place] = e < experts ? static_cast<int>(a) : -1;
    }
    __syncwarp();
  }
}

// --------------------------------------------------------------- moving rows
//
// A group of threads serves one token: it reads the token's row once and
// writes (or reads and sums) its k rows.  `log_group` threads a token, the
// block's 256 threads serving several narrow tokens or one wide one.
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

template <typename T, int V>
__global__ void __launch_bounds__(kMoveThreads)
    dispatch_kernel(const T* __restrict__ x, int64_t tokens, int k, int vecs, int64_t x_stride,
                    const int* __restrict__ offsets, int experts, const int* __restrict__ position,
                    T* __restrict__ rows, int64_t rows_stride, int log_group) {
  const Group g = my_group(log_group);
  if (g.token >= tokens) return;
  const int64_t all = tokens * k;
  const int* pos = position + g.token * k;
  const int64_t kept = kept_rows(offsets, experts, all);
  for (int c = g.t; c < vecs; c += g.size) {
    const Pack<T, V> v = *reinterpret_cast<const Pack<T, V>*>(x + g.token * x_stride + c * V);
    for (int j = 0; j < k; ++j) {
      const int64_t p = pos[j];
      if (p >= 0 && p < all)
        *reinterpret_cast<Pack<T, V>*>(rows + p * rows_stride + c * V) = v;
    }
  }
  // the rows of the dropped assignments: each token clears its own k places
  for (int64_t r = g.token * k < kept ? kept : g.token * k; r < (g.token + 1) * k; ++r)
    for (int c = g.t; c < vecs; c += g.size) {
      Pack<T, V> z;
#pragma unroll
      for (int i = 0; i < V; ++i) z.v[i] = from_f32<T>(0.f);
      *reinterpret_cast<Pack<T, V>*>(rows + r * rows_stride + c * V) = z;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kMoveThreads)
    combine_kernel(const T* __restrict__ y, int64_t tokens, int k, int vecs, int64_t y_stride,
                   const int* __restrict__ position, const float* __restrict__ weights,
                   T* __restrict__ out, int64_t out_stride, int log_group) {
  const Group g = my_group(log_group);
  if (g.token >= tokens) return;
  const int64_t all = tokens * k;
  const int* pos = position + g.token * k;
  const float* w = weights + g.token * k;
  for (int c = g.t; c < vecs; c += g.size) {
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int j = 0; j < k; ++j) {
      const int64_t p = pos[j];
      if (p < 0 || p >= all) continue;
      const float s = weights ? w[j] : 1.f;
      const Pack<T, V> v = *reinterpret_cast<const Pack<T, V>*>(y + p * y_stride + c * V);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(s, to_f32(v.v[i]), acc[i]);
    }
    Pack<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(acc[i]);
    *reinterpret_cast<Pack<T, V>*>(out + g.token * out_stride + c * V) = o;
  }
}

// One warp a token: the dot products are sums over the warp's lanes.
template <typename T, int V>
__global__ void __launch_bounds__(kMoveThreads)
    combine_backward_kernel(const T* __restrict__ grad_out, const T* __restrict__ y,
                            int64_t tokens, int k, int vecs, int64_t go_stride, int64_t y_stride,
                            const int* __restrict__ offsets, int experts,
                            const int* __restrict__ position, const float* __restrict__ weights,
                            T* __restrict__ grad_y, int64_t gy_stride,
                            float* __restrict__ grad_weights) {
  const Group g = my_group(5);
  if (g.token >= tokens) return;
  const int64_t all = tokens * k;
  const int* pos = position + g.token * k;
  const T* go = grad_out + g.token * go_stride;
  for (int j = 0; j < k; ++j) {
    const int64_t p = pos[j];
    const bool on = p >= 0 && p < all;
    float dot = 0.f;
    if (on) {
      const float s = weights ? weights[g.token * k + j] : 1.f;
      for (int c = g.t; c < vecs; c += 32) {
        const Pack<T, V> d = *reinterpret_cast<const Pack<T, V>*>(go + c * V);
        if (grad_weights) {
          const Pack<T, V> v = *reinterpret_cast<const Pack<T, V>*>(y + p * y_stride + c * V);
#pragma unroll
          for (int i = 0; i < V; ++i) dot = fmaf(to_f32(d.v[i]), to_f32(v.v[i]), dot);
        }
        if (grad_y) {
          Pack<T, V> o;
#pragma unroll
          for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(s * to_f32(d.v[i]));
          *reinterpret_cast<Pack<T, V>*>(grad_y + p * gy_stride + c * V) = o;
        }
      }
    }
    if (grad_weights) {
#pragma unroll
      for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
      if (g.t == 0) grad_weights[g.token * k + j] = dot;
    }
  }
  if (!grad_y) return;
  const int64_t kept = kept_rows(offsets, experts, all);
  for (int64_t r = g.token * k < kept ? kept : g.token * k; r < (g.token + 1) * k; ++r)
    for (int c = g.t; c < vecs; c += 32) {
      Pack<T, V> z;
#pragma unroll
      for (int i = 0; i < V; ++i) z.v[i] = from_f32<T>(0.f);
      *reinterpret_cast<Pack<T, V>*>(grad_y + r * gy_stride + c * V) = z;
    }
}

// -------------------------------------------------------------- host checks

tbe_status check_rows(int32_t dtype, int64_t tokens, int32_t k, int64_t width) {
  if (tokens < 0 || k < 1 || width < 0) return TBE_EINVAL;
  if (!dtype_bytes(dtype)) return TBE_EUNSUPPORTED;
  if (tokens > INT32_MAX / k || width > INT32_MAX) return TBE_EUNSUPPORTED;
  return TBE_OK;
}

bool check_matrix(const void* p, int32_t dtype, int64_t stride, int64_t width) {
  return p && stride >= width && aligned_to(p, dtype_bytes(dtype));
}

bool check_plan(const int32_t* offsets, const int32_t* position) {
  return offsets && position && aligned_to(offsets, 4) && aligned_to(position, 4);
}

// Whether rows starting at p, `stride` elements apart, can be moved in
// 16-byte vectors from end to end.
bool vector_rows(const void* p, int bytes, int64_t stride, int64_t width) {
  return aligned_to(p, 16) && stride * bytes % 16 == 0 && width * bytes % 16 == 0;
}

int log_group_of(int64_t vecs) {
  int lg = 0;
  while (lg < 8 && (1 << lg) < vecs) ++lg;
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

// Calls f with a value of the row type and the vector length as a constant.
template <int V>
struct VecTag {
  static constexpr int v = V;
};
template <typename F>
tbe_status for_dtype(int32_t dtype, bool vec, F f) {
  if (dtype == TBE_DT_F32) return vec ? f(float{}, VecTag<4>{}) : f(float{}, VecTag<1>{});
  if (dtype == TBE_DT_F16) return vec ? f(__half{}, VecTag<8>{}) : f(__half{}, VecTag<1>{});
  return vec ? f(__nv_bfloat16{}, VecTag<8>{}) : f(__nv_bfloat16{}, VecTag<1>{});
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
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int n = static_cast<int>(tokens * k);
  const size_t smem = static_cast<size_t>(kSortWarps) * (experts + 1) * 4;
  const auto go = [&](auto* p, auto kernel) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSortWarps * (TBE_MAX_EXPERTS + 1) * 4) != cudaSuccess)
      return TBE_ECUDA;
    kernel<<<1, kSortWarps * 32, smem, s>>>(p, n, experts, offsets, source, position);
    return launched();
  };
  return index_dtype == TBE_DT_I32
             ? go(static_cast<const int32_t*>(ids), expert_sort_kernel<int32_t>)
             : go(static_cast<const int64_t*>(ids), expert_sort_kernel<int64_t>);
}

extern "C" tbe_status tbe_expert_dispatch(const void* x, int32_t dtype, int64_t tokens, int32_t k,
                                          int64_t width, int64_t x_stride, const int32_t* offsets,
                                          int32_t experts, const int32_t* position, void* rows,
                                          int64_t rows_stride, void* stream) {
  const tbe_status bad = check_rows(dtype, tokens, k, width);
  if (bad != TBE_OK) return bad;
  if (!tokens || !width) return TBE_OK;
  if (experts < 1 || !check_plan(offsets, position) || !check_matrix(x, dtype, x_stride, width) ||
      !check_matrix(rows, dtype, rows_stride, width))
    return TBE_EINVAL;
  const int b = dtype_bytes(dtype);
  const bool vec = vector_rows(x, b, x_stride, width) && vector_rows(rows, b, rows_stride, width);
  return for_dtype(dtype, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::v;
    const int vecs = static_cast<int>(width / V), lg = log_group_of(vecs);
    dispatch_kernel<T, V><<<static_cast<unsigned>(group_blocks(tokens, lg)), kMoveThreads, 0,
                            static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(x), tokens, k, vecs, x_stride, offsets, experts, position,
        static_cast<T*>(rows), rows_stride, lg);
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
      !check_matrix(out, dtype, out_stride, width) || !aligned_to(weights, 4))
    return TBE_EINVAL;
  const int b = dtype_bytes(dtype);
  const bool vec = vector_rows(y, b, y_stride, width) && vector_rows(out, b, out_stride, width);
  return for_dtype(dtype, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::v;
    const int vecs = static_cast<int>(width / V), lg = log_group_of(vecs);
    combine_kernel<T, V><<<static_cast<unsigned>(group_blocks(tokens, lg)), kMoveThreads, 0,
                           static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(y), tokens, k, vecs, y_stride, position, weights,
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
  const int b = dtype_bytes(dtype);
  const bool vec = vector_rows(grad_out, b, grad_out_stride, width) &&
                   (!grad_weights || vector_rows(y, b, y_stride, width)) &&
                   (!grad_y || vector_rows(grad_y, b, grad_y_stride, width));
  return for_dtype(dtype, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::v;
    combine_backward_kernel<T, V><<<static_cast<unsigned>(group_blocks(tokens, 5)), kMoveThreads,
                                    0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(grad_out), static_cast<const T*>(y), tokens, k,
        static_cast<int>(width / V), grad_out_stride, y_stride, offsets, experts, position,
        weights, static_cast<T*>(grad_y), grad_y_stride, grad_weights);
    return launched();
  });
}
