// Global norm over many gradients, and clipping.  The operations are specified
// in include/tbe_grads.h.
//
// Both passes move bytes and compute next to nothing, so what bounds them is
// memory: the squares read every gradient once, the scaling reads and writes it
// once more.  The tensors' addresses travel in the launch's parameters, up to
// 1024 a launch.  A tensor is cut into chunks of 16 KB, counted from the 16-byte
// boundary at or before its first element, so that every vector inside is
// aligned whatever the tensor's own address; CTA b takes a run of consecutive
// chunks, four 16-byte loads in flight a thread.  Every CTA leaves one fp64 sum
// of squares, so the total's order depends on the sizes, on where in 16 bytes the
// tensors begin, and on nothing else.  The scaling walks each run backwards: what
// the squares read last is still in L2.  2^29 bf16 elements in 300 tensors: squares
// 160 us (6.7 TB/s), scaling 334 us (6.4 TB/s).
#include <type_traits>

#include "internal.h"
#include "rows.cuh"
#include "tbe_grads.h"

namespace tbe {
namespace {

constexpr int kGradThreads = 256;
constexpr int kVecsPerThread = 4;
constexpr int kChunkBytes = kGradThreads * kVecsPerThread * 16;
constexpr int kGradCtas = 152 * 8;  // as many as are resident
constexpr int kFlush = 4;           // chunks whose squares a thread sums in fp32
constexpr int kShortList = 64, kLongList = 1024;  // tensors of one launch
static_assert(kGradCtas * sizeof(double) <= TBE_GRAD_WORKSPACE_BYTES, "one sum a CTA");

template <int kMost>
struct GradList {
  const void* grad[kMost];
  void* out[kMost];
  uint64_t numel_type[kMost];   // elements, and the type from bit 56
  uint32_t chunk0[kMost + 1];   // first chunk of each tensor
  int32_t count;
  __device__ __forceinline__ int64_t numel(int t) const {
    return static_cast<int64_t>(numel_type[t] & 0xffffffffffffffull);
  }
  __device__ __forceinline__ int type(int t) const {
    return static_cast<int>(numel_type[t] >> 56);
  }
  // The tensor that holds `chunk`.
  __device__ __forceinline__ int tensor_of(uint32_t chunk) const {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (chunk0[mid] <= chunk) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

// This CTA's run of chunks.
template <int kMost>
__device__ __forceinline__ void my_run(const GradList<kMost>& L, uint32_t* first, uint32_t* last) {
  const uint64_t total = L.chunk0[L.count];
  *first = static_cast<uint32_t>(total * blockIdx.x / gridDim.x);
  *last = static_cast<uint32_t>(total * (blockIdx.x + 1) / gridDim.x);
}

template <typename F>
__device__ __forceinline__ void with_type(int type, F f) {
  if (type == TBE_DT_F32) f(float{});
  else if (type == TBE_DT_F16) f(__half{});
  else f(__nv_bfloat16{});
}

// One chunk's values of this thread, zeros outside the tensor.  `at`: the
// chunk's first element, counted from the boundary before the tensor.
template <typename T>
__device__ __forceinline__ void load_chunk(const T* g, int64_t numel, int64_t at,
                                           Pack<T, kVec<T>> (&v)[kVecsPerThread]) {
  constexpr int V = kVec<T>;
  const int shift = lead<T>(g);
  const T* base = g - shift + at;
  const int64_t lo = shift - at, hi = lo + numel;  // the tensor, from `base`
  if (lo <= 0 && hi >= kChunkBytes / static_cast<int>(sizeof(T))) {
#pragma unroll
    for (int i = 0; i < kVecsPerThread; ++i) {
      v[i] = reinterpret_cast<const Pack<T, V>*>(base)[i * kGradThreads + threadIdx.x];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVecsPerThread; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int64_t j = static_cast<int64_t>(i * kGradThreads + threadIdx.x) * V + e;
        v[i].v[e] = j >= lo && j < hi ? base[j] : from_f32<T>(0.f);
      }
  }
}

template <typename T>
__device__ __forceinline__ float sum_squares_of(
    const Pack<T, kVec<T>> (&v)[kVecsPerThread], float f) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kVecsPerThread; ++i) {
    float x[kVec<T>];
    to_floats<T>(v[i], x);
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) s = fmaf(x[e] * f, x[e] * f, s);
  }
  return s;
}

__device__ __forceinline__ double block_sum(double v, double* smem) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < kGradThreads / 32; ++i) s += smem[i];
  __syncthreads();
  return s;
}

template <int kMost>
__global__ void __launch_bounds__(kGradThreads)
    grad_squares_kernel(const __grid_constant__ GradList<kMost> L, double* __restrict__ partial,
                        bool first_list) {
  __shared__ double smem[kGradThreads / 32];
  uint32_t chunk, last;
  my_run(L, &chunk, &last);
  double sum = 0.0;
  float run = 0.f;
  int held = 0;
  int t = chunk < last ? L.tensor_of(chunk) : 0;
  for (; chunk < last; ++chunk) {
    while (chunk >= L.chunk0[t + 1]) ++t;
    with_type(L.type(t), [&](auto tag) {
      using T = decltype(tag);
      Pack<T, kVec<T>> v[kVecsPerThread];
      load_chunk<T>(static_cast<const T*>(L.grad[t]), L.numel(t),
                    static_cast<int64_t>(chunk - L.chunk0[t]) * (kChunkBytes / sizeof(T)), v);
      const float s = sum_squares_of<T>(v, 1.f);
      // Outside the range in which no square that counts is lost, the sum is formed again with
      // the values times 2^80 or 2^-80.  (Zeros and NaN come out as they are.)
      if (s > 0x1p100f)
        sum += static_cast<double>(sum_squares_of<T>(v, 0x1p-80f)) * 0x1p160;
      else if (s < 0x1p-60f)
        sum += static_cast<double>(sum_squares_of<T>(v, 0x1p80f)) * 0x1p-160;
      else
        run += s;
    });
    if (++held == kFlush) {
      sum += static_cast<double>(run);
      run = 0.f;
      held = 0;
    }
  }
  sum += static_cast<double>(run);
  sum = block_sum(sum, smem);
  if (threadIdx.x == 0) partial[blockIdx.x] = first_list ? sum : partial[blockIdx.x] + sum;
}

__device__ __forceinline__ float total_norm(const double* partial, int ctas, double* smem) {
  double s = 0.0;
  for (int i = threadIdx.x; i < ctas; i += kGradThreads) s += partial[i];
  return static_cast<float>(sqrt(block_sum(s, smem)));
}

__global__ void __launch_bounds__(kGradThreads)
    grad_norm_kernel(const double* __restrict__ partial, int ctas, float* __restrict__ norm) {
  __shared__ double smem[kGradThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float n = total_norm(partial, ctas, smem);
  if (threadIdx.x == 0) *norm = n;
}

template <int kMost>
__global__ void __launch_bounds__(kGradThreads)
    grad_scale_kernel(const __grid_constant__ GradList<kMost> L,
                      const double* __restrict__ partial, int ctas, float max_norm,
                      float* __restrict__ norm) {
  __shared__ double smem[kGradThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float n = total_norm(partial, ctas, smem);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float q = __fdiv_rn(max_norm, n + 1e-6f);
  const float c = q > 1.f ? 1.f : q;  // a NaN stays one
  uint32_t first, chunk;
  my_run(L, &first, &chunk);
  int t = first < chunk ? L.tensor_of(chunk - 1) : 0;
  while (chunk-- > first) {
    while (chunk < L.chunk0[t]) --t;
    if (c == 1.f && L.out[t] == L.grad[t]) continue;
    with_type(L.type(t), [&](auto tag) {
      using T = decltype(tag);
      constexpr int V = kVec<T>;
      const T* g = static_cast<const T*>(L.grad[t]);
      T* out = static_cast<T*>(L.out[t]);
      const int64_t numel = L.numel(t);
      const int64_t at =
          static_cast<int64_t>(chunk - L.chunk0[t]) * (kChunkBytes / static_cast<int>(sizeof(T)));
      Pack<T, V> v[kVecsPerThread];
      load_chunk<T>(g, numel, at, v);
#pragma unroll
      for (int i = 0; i < kVecsPerThread; ++i) {
        float x[V];
        to_floats<T>(v[i], x);
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] *= c;
        v[i] = from_floats<T>(x);
      }
      const int shift = lead<T>(g);
      const int64_t lo = shift - at, hi = lo + numel;
      T* base = out - shift + at;
      const bool whole = lo <= 0 && hi >= kChunkBytes / static_cast<int>(sizeof(T));
      if (whole && lead<T>(out) == shift) {
#pragma unroll
        for (int i = 0; i < kVecsPerThread; ++i)
          reinterpret_cast<Pack<T, V>*>(base)[i * kGradThreads + threadIdx.x] = v[i];
      } else {
#pragma unroll
        for (int i = 0; i < kVecsPerThread; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const int64_t j = static_cast<int64_t>(i * kGradThreads + threadIdx.x) * V + e;
            if (j >= lo && j < hi) base[j] = v[i].v[e];
          }
      }
    });
  }
}

tbe_status check_grads(const tbe_grad_tensor* tensors, int64_t count, const float* norm,
                       const void* ws, size_t ws_bytes, bool clip) {
  if (count < 0 || (count && !tensors) || !norm || !aligned_to(norm, 4)) return TBE_EINVAL;
  for (int64_t i = 0; i < count; ++i) {
    const tbe_grad_tensor& t = tensors[i];
    const int b = dtype_bytes(t.dtype);
    if (t.numel < 0) return TBE_EINVAL;
    if (!b || t.numel > (int64_t(1) << 40)) return TBE_EUNSUPPORTED;
    if (t.numel && (!t.grad || !aligned_to(t.grad, b))) return TBE_EINVAL;
    if (t.numel && clip && (!t.out || !aligned_to(t.out, b))) return TBE_EINVAL;
  }
  if (!ws || ws_bytes < TBE_GRAD_WORKSPACE_BYTES || !aligned_to(ws, 16)) return TBE_EWORKSPACE;
  return TBE_OK;
}

int64_t chunks_of(const tbe_grad_tensor& t) {
  if (!t.numel) return 0;
  const int64_t b = dtype_bytes(t.dtype);
  const int64_t shift = (reinterpret_cast<uintptr_t>(t.grad) & 15) / b;
  return ((t.numel + shift) * b + kChunkBytes - 1) / kChunkBytes;
}

// Calls f(list) for the tensors with elements, at most kMost at a time.
template <int kMost, typename F>
tbe_status for_lists(const tbe_grad_tensor* tensors, int64_t count, F f) {
  GradList<kMost> L;
  L.count = 0;
  L.chunk0[0] = 0;
  for (int64_t i = 0; i < count; ++i) {
    const tbe_grad_tensor& t = tensors[i];
    const int64_t chunks = chunks_of(t);
    if (!chunks) continue;
    if (L.count == kMost || L.chunk0[L.count] + chunks > INT32_MAX) {
      const tbe_status st = f(L);
      if (st != TBE_OK) return st;
      L.count = 0;
    }
    const int c = L.count++;
    L.grad[c] = t.grad;
    L.out[c] = t.out;
    L.numel_type[c] = static_cast<uint64_t>(t.numel) | static_cast<uint64_t>(t.dtype) << 56;
    L.chunk0[c + 1] = static_cast<uint32_t>(L.chunk0[c] + chunks);
  }
  return L.count ? f(L) : TBE_OK;
}

int ctas_for(const tbe_grad_tensor* tensors, int64_t count) {
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) chunks += chunks_of(tensors[i]);
  return static_cast<int>(chunks < kGradCtas ? chunks : kGradCtas);
}

// A launch that may begin before the kernel ahead of it ends; the kernel waits
// for that one's results itself (griddepcontrol.wait).
template <typename... Args>
tbe_status launch_after(void (*kernel)(Args...), int ctas, cudaStream_t s,
                        std::common_type_t<Args>... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kGradThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return TBE_ECUDA;
  note_launch();
  return TBE_OK;
}

template <int kMost>
tbe_status norm_and_clip(const tbe_grad_tensor* tensors, int64_t count, bool clip, float max_norm,
                         float* norm, double* partial, cudaStream_t s) {
  const int ctas = ctas_for(tensors, count);
  bool first = true;
  tbe_status st = for_lists<kMost>(tensors, count, [&](const GradList<kMost>& L) {
    grad_squares_kernel<kMost><<<ctas, kGradThreads, 0, s>>>(L, partial, first);
    note_launch();
    first = false;
    return cudaGetLastError() == cudaSuccess ? TBE_OK : TBE_ECUDA;
  });
  if (st != TBE_OK) return st;
  if (!clip || !ctas) return launch_after(grad_norm_kernel, 1, s, partial, ctas, norm);
  return for_lists<kMost>(tensors, count, [&](const GradList<kMost>& L) {
    return launch_after(grad_scale_kernel<kMost>, ctas, s, L, partial, ctas, max_norm, norm);
  });
}

tbe_status run_grads(const tbe_grad_tensor* tensors, int64_t count, bool clip, float max_norm,
                     float* norm, void* workspace, size_t ws_bytes, void* stream) {
  const tbe_status bad = check_grads(tensors, count, norm, workspace, ws_bytes, clip);
  if (bad != TBE_OK) return bad;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  // a launch copies its parameters: 1.9 KB for a short list, 29 KB for a long one
  if (count <= kShortList)
    return norm_and_clip<kShortList>(tensors, count, clip, max_norm, norm, partial, s);
  return norm_and_clip<kLongList>(tensors, count, clip, max_norm, norm, partial, s);
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_grad_norm(const tbe_grad_tensor* tensors, int64_t count, float* norm,
                                    void* workspace, size_t ws_bytes, void* stream) {
  return run_grads(tensors, count, false, 0.f, norm, workspace, ws_bytes, stream);
}

extern "C" tbe_status tbe_grad_clip(const tbe_grad_tensor* tensors, int64_t count, float max_norm,
                                    float* norm, void* workspace, size_t ws_bytes, void* stream) {
  if (!(max_norm >= 0.f)) return TBE_EINVAL;
  return run_grads(tensors, count, true, max_norm, norm, workspace, ws_bytes, stream);
}
