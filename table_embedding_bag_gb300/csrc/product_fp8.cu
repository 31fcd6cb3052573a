// 8-bit rows and weights with a scale for each block of 128, and the experts'
// products on them.  The operations are specified in include/tbe_experts.h.
#include <cuda_fp8.h>

#include "internal.h"
#include "rows.cuh"
#include "tbe_experts.h"

namespace tbe {
namespace {

constexpr int kBlock = TBE_SCALE_BLOCK;
constexpr float kInvMax = 1.f / 448.f;  // one over the largest e4m3 value, rounded to fp32
constexpr float kTinyScale = 0x1p-126f;

__device__ __forceinline__ float block_scale(float amax) {
  return fmaxf(amax * kInvMax, kTinyScale);
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float from_e4m3(uint8_t v) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

// One warp a sorted place's source row and block of 128 columns: the row is read
// once, its 4 values a lane stay in registers, and all its k places are
// written.
template <typename T>
__global__ void __launch_bounds__(256)
    dispatch_fp8_kernel(const T* __restrict__ x, int64_t tokens, int k, int64_t width,
                        int64_t x_stride, const int* __restrict__ offsets, int experts,
                        const int* __restrict__ position, uint8_t* __restrict__ q,
                        int64_t q_stride, float* __restrict__ scale) {
  const int blocks = static_cast<int>((width + kBlock - 1) / kBlock);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (unit >= tokens * blocks) return;
  const int lane = threadIdx.x & 31;
  const int64_t token = unit / blocks;
  const int b = static_cast<int>(unit % blocks);
  const int64_t col = static_cast<int64_t>(b) * kBlock + lane * 4;
  float v[4];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = col + i < width ? to_f32(x[token * x_stride + col + i]) : 0.f;
    amax = fmaxf(amax, fabsf(v[i]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = block_scale(amax);
  uint8_t e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = to_e4m3(__fdiv_rn(v[i], s));
  const int64_t all = tokens * k;
  for (int j = 0; j < k; ++j) {
    const int64_t p = position ? position[token * k + j] : token;
    if (p < 0 || p >= all) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < width) q[p * q_stride + col + i] = e[i];
    if (lane == 0) scale[p * blocks + b] = s;
  }
  if (!position) return;
  int64_t kept = offsets[experts];
  kept = kept < 0 ? 0 : kept > all ? all : kept;
  for (int64_t r = token * k < kept ? kept : token * k; r < (token + 1) * k; ++r) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < width) q[r * q_stride + col + i] = 0;
    if (lane == 0) scale[r * blocks + b] = kTinyScale;
  }
}

// One CTA a 128 x 128 block of an expert's weights.
template <typename T>
__global__ void __launch_bounds__(256)
    quantize_weights_kernel(const T* __restrict__ w, int64_t n, int64_t k, int nb, int kb,
                            uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ float warp_max[8];
  const int64_t unit = blockIdx.x;
  const int64_t e = unit / (static_cast<int64_t>(nb) * kb);
  const int64_t row0 = unit / kb % nb * kBlock, col0 = unit % kb * kBlock;
  const T* src = w + e * n * k;
  uint8_t* dst = q + e * n * k;
  const int c = threadIdx.x & (kBlock - 1);
  const bool in = col0 + c < k;
  float amax = 0.f;
  for (int r = threadIdx.x / kBlock; r < kBlock && row0 + r < n; r += 256 / kBlock)
    if (in) amax = fmaxf(amax, fabsf(to_f32(src[(row0 + r) * k + col0 + c])));
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, warp_max[i]);
  const float s = block_scale(amax);
  for (int r = threadIdx.x / kBlock; r < kBlock && row0 + r < n; r += 256 / kBlock)
    if (in)
      dst[(row0 + r) * k + col0 + c] =
          to_e4m3(__fdiv_rn(to_f32(src[(row0 + r) * k + col0 + c]), s));
  if (threadIdx.x == 0) scale[unit] = s;
}

// ------------------------------------------------------------------- product
//
// A CTA owns 64 output rows x 64 columns of one expert; a thread 4 x 4 of
// them.  A grid row of row tiles is walked over the experts by every CTA.
constexpr int kTile = 64, kStep = 32;

__device__ __forceinline__ int clamp_offset(const int* offsets, int e, int rows) {
  const int v = offsets[e];
  return v < 0 ? 0 : v > rows ? rows : v;
}

template <typename T>
__global__ void __launch_bounds__(256)
    product_kernel(const uint8_t* __restrict__ a, int64_t a_stride,
                   const float* __restrict__ a_scale, const uint8_t* __restrict__ w,
                   const float* __restrict__ w_scale, const int* __restrict__ offsets, int rows,
                   int64_t n, int64_t k, int experts, T* __restrict__ out, int64_t out_stride) {
  __shared__ float sa[kStep][kTile + 1], sw[kStep][kTile + 1];
  const int kb = static_cast<int>((k + kBlock - 1) / kBlock);
  const int nb = static_cast<int>((n + kBlock - 1) / kBlock);
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int tr = threadIdx.x / 16 * 4, tc = threadIdx.x % 16 * 4;
  int tile = blockIdx.x, start = 0;
  for (int e = 0; e <= experts; ++e) {  // e == experts: the rows past the last expert
    int end = rows;
    if (e < experts && offsets) {
      end = clamp_offset(offsets, e + 1, rows);
      if (e == 0) start = clamp_offset(offsets, 0, rows);
      if (end < start) end = start;
    }
    const int tiles = (end - start + kTile - 1) / kTile;
    for (; tile < tiles; tile += gridDim.x) {
      const int r0 = start + tile * kTile;
      float acc[4][4] = {};
      for (int b = 0; b < kb && e < experts; ++b) {
        float part[4][4] = {};
        for (int64_t k0 = static_cast<int64_t>(b) * kBlock; k0 < k && k0 < (b + 1) * kBlock;
             k0 += kStep) {
          __syncthreads();
          for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
            const int r = i / kStep, c = i % kStep;
            sa[c][r] = r0 + r < end && k0 + c < k ? from_e4m3(a[(r0 + r) * a_stride + k0 + c]) : 0.f;
            sw[c][r] = n0 + r < n && k0 + c < k ? from_e4m3(w[(e * n + n0 + r) * k + k0 + c]) : 0.f;
          }
          __syncthreads();
          for (int c = 0; c < kStep; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[c][tr + i], sw[c][tc + j], part[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (r0 + tr + i >= end || n0 + tc >= n) continue;
          const float s = a_scale[static_cast<int64_t>(r0 + tr + i) * kb + b] *
                          w_scale[(static_cast<int64_t>(e) * nb + (n0 + tc) / kBlock) * kb + b];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s, part[i][j], acc[i][j]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r0 + tr + i < end && n0 + tc + j < n)
            out[(r0 + tr + i) * out_stride + n0 + tc + j] = from_f32<T>(acc[i][j]);
    }
    tile -= tiles;
    start = end;
  }
}

tbe_status launched() {
  note_launch();
  return cudaGetLastError() == cudaSuccess ? TBE_OK : TBE_ECUDA;
}

template <typename F>
tbe_status for_dtype(int32_t dtype, F f) {
  if (dtype == TBE_DT_F32) return f(float{});
  if (dtype == TBE_DT_F16) return f(__half{});
  return f(__nv_bfloat16{});
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_expert_dispatch_fp8(const void* x, int32_t dtype, int64_t tokens,
                                              int32_t k, int64_t width, int64_t x_stride,
                                              const int32_t* offsets, int32_t experts,
                                              const int32_t* position, uint8_t* q,
                                              int64_t q_stride, float* scale, void* stream) {
  if (tokens < 0 || k < 1 || width < 0) return TBE_EINVAL;
  if (!dtype_bytes(dtype)) return TBE_EUNSUPPORTED;
  if (tokens > INT32_MAX / k || width > INT32_MAX) return TBE_EUNSUPPORTED;
  if (!tokens || !width) return TBE_OK;
  if (position ? (experts < 1 || !offsets || !aligned_to(offsets, 4) || !aligned_to(position, 4))
               : k != 1)
    return TBE_EINVAL;
  if (!x || !q || !scale || x_stride < width || q_stride < width ||
      !aligned_to(x, dtype_bytes(dtype)) || !aligned_to(scale, 4))
    return TBE_EINVAL;
  const int64_t units = tokens * ((width + kBlock - 1) / kBlock);
  if ((units + 7) / 8 > INT32_MAX) return TBE_EUNSUPPORTED;
  return for_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    dispatch_fp8_kernel<T><<<static_cast<unsigned>((units + 7) / 8), 256, 0,
                             static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(x), tokens, k, width, x_stride, offsets, experts, position, q,
        q_stride, scale);
    return launched();
  });
}

extern "C" tbe_status tbe_quantize_weights(const void* w, int32_t dtype, int64_t experts,
                                           int64_t n, int64_t k, uint8_t* q, float* scale,
                                           void* stream) {
  if (experts < 0 || n < 0 || k < 0) return TBE_EINVAL;
  if (!dtype_bytes(dtype)) return TBE_EUNSUPPORTED;
  if (n > INT32_MAX || k > INT32_MAX || experts > INT32_MAX) return TBE_EUNSUPPORTED;
  if (!experts || !n || !k) return TBE_OK;
  if (!w || !q || !scale || !aligned_to(w, dtype_bytes(dtype)) || !aligned_to(scale, 4))
    return TBE_EINVAL;
  const int64_t nb = (n + kBlock - 1) / kBlock, kb = (k + kBlock - 1) / kBlock;
  if (nb * kb > INT32_MAX / experts) return TBE_EUNSUPPORTED;
  return for_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    quantize_weights_kernel<T><<<static_cast<unsigned>(experts * nb * kb), 256, 0,
                                 static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(w), n, k, static_cast<int>(nb), static_cast<int>(kb), q, scale);
    return launched();
  });
}

extern "C" tbe_status tbe_expert_product(const uint8_t* a, int64_t a_stride, const float* a_scale,
                                         const uint8_t* w, const float* w_scale,
                                         const int32_t* offsets, int64_t rows, int64_t n,
                                         int64_t k, int32_t experts, void* out, int32_t out_dtype,
                                         int64_t out_stride, int32_t* status, void* stream) {
  (void)status;
  if (rows < 0 || n < 0 || k < 1 || experts < 1) return TBE_EINVAL;
  if (!dtype_bytes(out_dtype)) return TBE_EUNSUPPORTED;
  if (rows > INT32_MAX || n > INT32_MAX || k > INT32_MAX || experts > TBE_MAX_EXPERTS ||
      experts * n > INT32_MAX)
    return TBE_EUNSUPPORTED;
  if (!rows || !n) return TBE_OK;
  if (!a || !a_scale || !w || !w_scale || !out || (!offsets && experts != 1) || a_stride < k ||
      out_stride < n)
    return TBE_EINVAL;
  if (!aligned_to(a_scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(offsets, 4) ||
      !aligned_to(out, dtype_bytes(out_dtype)))
    return TBE_EINVAL;
  if (k % 16 || a_stride % 16 || !aligned_to(a, 16) || !aligned_to(w, 16)) return TBE_EUNSUPPORTED;
  if ((n + kTile - 1) / kTile > 65535) return TBE_EUNSUPPORTED;
  return for_dtype(out_dtype, [&](auto t) {
    using T = decltype(t);
    const dim3 grid(static_cast<unsigned>(rows / kTile + 1 < 1024 ? rows / kTile + 1 : 1024),
                    static_cast<unsigned>((n + kTile - 1) / kTile));
    product_kernel<T><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        a, a_stride, a_scale, w, w_scale, offsets, static_cast<int>(rows), n, k, experts,
        static_cast<T*>(out), out_stride);
    return launched();
  });
}
