// Global norm over many gradients, and clipping.  The operations are specified
// in include/tbe_grads.h.
//
// The tensors' addresses travel in the launch's parameters, up to kMaxList a
// launch; the tensors are cut into chunks of kChunkElems elements, and CTA b
// takes chunks b, b + gridDim.x, ... of the list.  Every CTA leaves one fp64
// sum of squares, so the total's order depends on the sizes alone.
#include <type_traits>

#include "internal.h"
#include "rows.cuh"
#include "tbe_grads.h"

namespace tbe {
namespace {

constexpr int kGradThreads = 256;
constexpr int kChunkElems = 8192;
constexpr int kPerThread = kChunkElems / kGradThreads;
constexpr int kMaxList = 128;   // tensors of one launch
constexpr int kGradCtas = 608;  // four a multiprocessor
static_assert(kGradCtas * sizeof(double) <= TBE_GRAD_WORKSPACE_BYTES, "one sum a CTA");

struct GradList {
  const void* grad[kMaxList];
  void* out[kMaxList];
  int64_t numel[kMaxList];
  int64_t chunk0[kMaxList + 1];  // first chunk of each tensor
  int32_t dtype[kMaxList];
  int32_t count;
};

// The list's tensor that holds `chunk`.
__device__ __forceinline__ int tensor_of(const GradList& L, int64_t chunk) {
  int lo = 0, hi = L.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (L.chunk0[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
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

// Sum of squares of up to kPerThread values in fp32.  Where it leaves the
// range in which no square that counts is lost, it is formed again with the
// values times 2^80 or 2^-80; the caller adds s * unscale in fp64.
__device__ __forceinline__ double squares(const float (&v)[kPerThread], int n) {
  float s = 0.f;
  for (int i = 0; i < kPerThread; ++i)
    if (i < n) s = fmaf(v[i], v[i], s);
  const float f = s > 0x1p100f ? 0x1p-80f : s < 0x1p-60f ? 0x1p80f : 1.f;
  if (f == 1.f) return s;
  float t = 0.f;
  for (int i = 0; i < kPerThread; ++i)
    if (i < n) t = fmaf(v[i] * f, v[i] * f, t);
  return static_cast<double>(t) * (f < 1.f ? 0x1p160 : 0x1p-160);
}

template <typename F>
__device__ __forceinline__ void with_type(int32_t dtype, F f) {
  if (dtype == TBE_DT_F32) f(float{});
  else if (dtype == TBE_DT_F16) f(__half{});
  else f(__nv_bfloat16{});
}

__global__ void __launch_bounds__(kGradThreads)
    grad_squares_kernel(const __grid_constant__ GradList L, double* __restrict__ partial,
                        bool first) {
  __shared__ double smem[kGradThreads / 32];
  double sum = 0.0;
  for (int64_t chunk = blockIdx.x; chunk < L.chunk0[L.count]; chunk += gridDim.x) {
    const int t = tensor_of(L, chunk);
    const int64_t at = (chunk - L.chunk0[t]) * kChunkElems;
    const int64_t left = L.numel[t] - at;
    with_type(L.dtype[t], [&](auto tag) {
      using T = decltype(tag);
      const T* g = static_cast<const T*>(L.grad[t]) + at;
      float v[kPerThread];
      for (int i = 0; i < kPerThread; ++i) {
        const int e = i * kGradThreads + threadIdx.x;
        v[i] = e < left ? to_f32(g[e]) : 0.f;
      }
      sum += squares(v, kPerThread);
    });
  }
  sum = block_sum(sum, smem);
  if (threadIdx.x == 0) partial[blockIdx.x] = first ? sum : partial[blockIdx.x] + sum;
}

__device__ __forceinline__ float total_norm(const double* partial, int ctas, double* smem) {
  double s = 0.0;
  for (int i = threadIdx.x; i < ctas; i += kGradThreads) s += partial[i];
  return static_cast<float>(sqrt(block_sum(s, smem)));
}

__global__ void __launch_bounds__(kGradThreads)
    grad_norm_kernel(const double* __restrict__ partial, int ctas, float* __restrict__ norm) {
  __shared__ double smem[kGradThreads / 32];
  const float n = total_norm(partial, ctas, smem);
  if (threadIdx.x == 0) *norm = n;
}

__global__ void __launch_bounds__(kGradThreads)
    grad_scale_kernel(const __grid_constant__ GradList L, const double* __restrict__ partial,
                      int ctas, float max_norm, float* __restrict__ norm) {
  __shared__ double smem[kGradThreads / 32];
  const float n = total_norm(partial, ctas, smem);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float q = __fdiv_rn(max_norm, n + 1e-6f);
  const float c = q > 1.f ? 1.f : q;  // a NaN stays one
  for (int64_t chunk = blockIdx.x; chunk < L.chunk0[L.count]; chunk += gridDim.x) {
    const int t = tensor_of(L, chunk);
    if (c == 1.f && L.out[t] == L.grad[t]) continue;
    const int64_t at = (chunk - L.chunk0[t]) * kChunkElems;
    const int64_t left = L.numel[t] - at;
    with_type(L.dtype[t], [&](auto tag) {
      using T = decltype(tag);
      const T* g = static_cast<const T*>(L.grad[t]) + at;
      T* o = static_cast<T*>(L.out[t]) + at;
      for (int e = threadIdx.x; e < kChunkElems && e < left; e += kGradThreads)
        o[e] = from_f32<T>(c * to_f32(g[e]));
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

// Calls f(list) for the tensors with elements, kMaxList at a time.
template <typename F>
tbe_status for_lists(const tbe_grad_tensor* tensors, int64_t count, F f) {
  GradList L;
  L.count = 0;
  L.chunk0[0] = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (!tensors[i].numel) continue;
    const int c = L.count++;
    L.grad[c] = tensors[i].grad;
    L.out[c] = tensors[i].out;
    L.numel[c] = tensors[i].numel;
    L.dtype[c] = tensors[i].dtype;
    L.chunk0[c + 1] = L.chunk0[c] + (tensors[i].numel + kChunkElems - 1) / kChunkElems;
    if (L.count == kMaxList) {
      const tbe_status st = f(L);
      if (st != TBE_OK) return st;
      L.count = 0;
    }
  }
  return L.count ? f(L) : TBE_OK;
}

int ctas_for(const tbe_grad_tensor* tensors, int64_t count) {
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i)
    chunks += (tensors[i].numel + kChunkElems - 1) / kChunkElems;
  return static_cast<int>(chunks < kGradCtas ? chunks : kGradCtas);
}

tbe_status launched() {
  note_launch();
  return cudaGetLastError() == cudaSuccess ? TBE_OK : TBE_ECUDA;
}

tbe_status sum_squares(const tbe_grad_tensor* tensors, int64_t count, int ctas, double* partial,
                       cudaStream_t s) {
  bool first = true;
  return for_lists(tensors, count, [&](const GradList& L) {
    grad_squares_kernel<<<ctas, kGradThreads, 0, s>>>(L, partial, first);
    first = false;
    return launched();
  });
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_grad_norm(const tbe_grad_tensor* tensors, int64_t count, float* norm,
                                    void* workspace, size_t ws_bytes, void* stream) {
  const tbe_status bad = check_grads(tensors, count, norm, workspace, ws_bytes, false);
  if (bad != TBE_OK) return bad;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  const int ctas = ctas_for(tensors, count);
  const tbe_status st = sum_squares(tensors, count, ctas, partial, s);
  if (st != TBE_OK) return st;
  grad_norm_kernel<<<1, kGradThreads, 0, s>>>(partial, ctas, norm);
  return launched();
}

extern "C" tbe_status tbe_grad_clip(const tbe_grad_tensor* tensors, int64_t count, float max_norm,
                                    float* norm, void* workspace, size_t ws_bytes, void* stream) {
  if (!(max_norm >= 0.f)) return TBE_EINVAL;
  const tbe_status bad = check_grads(tensors, count, norm, workspace, ws_bytes, true);
  if (bad != TBE_OK) return bad;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  const int ctas = ctas_for(tensors, count);
  if (!ctas) return tbe_grad_norm(tensors, count, norm, workspace, ws_bytes, stream);
  const tbe_status st = sum_squares(tensors, count, ctas, partial, s);
  if (st != TBE_OK) return st;
  return for_lists(tensors, count, [&](const GradList& L) {
    grad_scale_kernel<<<ctas, kGradThreads, 0, s>>>(L, partial, ctas, max_norm, norm);
    return launched();
  });
}
