// Root-mean-square norm with the residual's addition, in the rows' type or in
// 8 bits, and its gradients.  The operations are specified in include/tbe_norm.h.
//
// A row is read once into the registers of the threads that share it (32 to 512 of them), its
// squares are summed, and its outputs are formed from the registers: memory bounds both
// directions.
#include <cmath>
#include <type_traits>

#include "entry.cuh"
#include "quantize.cuh"
#include "tbe_norm.h"

namespace tbe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kNormThreads = 512;     // threads of a CTA, at most
constexpr int kNormCta = 256;         // and as a rule
constexpr int kNormParts = 152 * 8;   // partial sums of grad_weight, at most
constexpr int kSumSegments = 32;

struct NormArgs {
  const void *x, *residual, *weight;
  void *h, *y;
  float* scale;
  int64_t xs, rs, hs, ys;
  int rows, width;
  bool w32;  // the weight is fp32
  float eps;
};

// Columns of unit j of this thread: vectors side by side, or single elements so that a
// warp's four consecutive units fill a block of 128 columns.
template <typename T, bool kAligned>
struct Units {
  static constexpr int V = kAligned ? kVec<T> : 1;
  static __device__ __forceinline__ int col(int j) {
    if constexpr (kAligned) return (j * static_cast<int>(blockDim.x) + threadIdx.x) * V;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    return ((j >> 2) * warps + warp) * kBlock + (j & 3) * 32 + lane;
  }
};

template <typename T, int V>
__device__ __forceinline__ void unit_floats(const Pack<T, V>& p, float (&f)[V]) {
  if constexpr (V == 1) f[0] = to_f32(p.v[0]);
  else to_floats<T>(p, f);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> unit_of(const float (&f)[V]) {
  if constexpr (V == 1) return {from_f32<T>(f[0])};
  else return from_floats<T>(f);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_unit(const T* row, int col, bool on) {
  if (on) return *reinterpret_cast<const Pack<T, V>*>(row + col);
  float zero[V] = {};
  return unit_of<T, V>(zero);
}
template <typename T, int V>
__device__ __forceinline__ void store_unit(T* row, int col, const Pack<T, V>& p) {
  *reinterpret_cast<Pack<T, V>*>(row + col) = p;
}

template <typename T, int V>
__device__ __forceinline__ void load_weight(const void* weight, bool w32, int col, bool on,
                                            float (&w)[V]) {
  if (!weight || !on) {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = 1.f;
  } else if (sizeof(T) == 4 || w32) {
    const float* p = static_cast<const float*>(weight) + col;
    if constexpr (V == 1) {
      w[0] = *p;
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(p + i);
        w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
      }
    }
  } else {
    unit_floats<T, V>(load_unit<T, V>(static_cast<const T*>(weight), col, true), w);
  }
}

// Sums over the threads of a row; the whole CTA calls it.  `part` has room for the CTA's warps.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*part)[N]) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kAll, v[i], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  float(*mine)[N] = part + threadIdx.y * warps;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) mine[threadIdx.x >> 5][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += mine[w][i];
}

template <typename T, bool kFp8, bool kAligned, int NV>
__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const NormArgs P) {
  using U = Units<T, kAligned>;
  constexpr int V = U::V;
  __shared__ float part[kNormThreads / 32][1];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = row < P.rows;  // the others take part in the barriers
  const T* x = static_cast<const T*>(P.x) + row * P.xs;
  Pack<T, V> v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) v[j] = load_unit<T, V>(x, U::col(j), live && U::col(j) < P.width);
  if (P.residual) {
    const T* r = static_cast<const T*>(P.residual) + row * P.rs;
    T* h = static_cast<T*>(P.h) + row * P.hs;
    Pack<T, V> b[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) b[j] = load_unit<T, V>(r, U::col(j), live && U::col(j) < P.width);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V], g[V];
      unit_floats<T, V>(v[j], f);
      unit_floats<T, V>(b[j], g);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] += g[i];
      v[j] = unit_of<T, V>(f);  // the sum as it is held
      if (P.h && live && U::col(j) < P.width) store_unit<T, V>(h, U::col(j), v[j]);
    }
  }
  float sum[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[V];
    unit_floats<T, V>(v[j], f);
#pragma unroll
    for (int i = 0; i < V; ++i) sum[0] = fmaf(f[i], f[i], sum[0]);
  }
  row_sums(sum, part);
  const float u = rsqrtf(__fdiv_rn(sum[0], static_cast<float>(P.width)) + P.eps);
  if constexpr (!kFp8) {
    T* y = static_cast<T*>(P.y) + row * P.ys;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = U::col(j);
      if (!live || col >= P.width) continue;
      float f[V], w[V];
      unit_floats<T, V>(v[j], f);
      load_weight<T, V>(P.weight, P.w32, col, true, w);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = f[i] * u * w[i];
      store_unit<T, V>(y, col, unit_of<T, V>(f));
    }
  } else {
    constexpr int kUnits = kAligned ? 1 : 4;          // units of a thread in a block of 128
    constexpr int kLanes = kAligned ? kBlock / V : 32;  // lanes that share it
    uint8_t* q = static_cast<uint8_t*>(P.y) + row * P.ys;
    float* scale = P.scale + row * ((P.width + kBlock - 1) / kBlock);
#pragma unroll
    for (int j = 0; j < NV; j += kUnits) {
      float f[kUnits * V];
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int col = U::col(j + k);
        float g[V], w[V];
        unit_floats<T, V>(v[j + k], g);
        load_weight<T, V>(P.weight, P.w32, col, col < P.width, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float y = live && col < P.width ? g[i] * u * w[i] : 0.f;
          f[k * V + i] = y;
          amax = fmaxf(amax, fabsf(y));  // passes over NaN
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
      const float s = block_scale(amax);
      const auto e = quantized(f, s);
      const int col = U::col(j);
      const int first = col - (threadIdx.x % kLanes) * V;  // of the block
      if (!live || first >= P.width) continue;
      if constexpr (kAligned) {
        if (col < P.width) *reinterpret_cast<Pack<uint8_t, V>*>(q + col) = e;
      } else {
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
          if (U::col(j + k) < P.width) q[U::col(j + k)] = e.v[k];
      }
      if (threadIdx.x % kLanes == 0) scale[first / kBlock] = s;
    }
  }
}

struct NormGradArgs {
  const void *gy, *h, *weight, *gh;
  void* gx;
  float* partial;  // [parts][width], or null
  int64_t gys, hs, ghs, gxs;
  int rows, width;
  bool w32;
  float eps;
};

// A group of threads walks rows a grid apart and keeps its columns' part of
// grad_weight in registers.
template <typename T, bool kAligned, int NV>
__global__ void __launch_bounds__(kNormThreads) rms_norm_backward_kernel(const NormGradArgs P) {
  using U = Units<T, kAligned>;
  constexpr int V = U::V;
  __shared__ float parts[2][kNormThreads / 32][2];
  float acc[NV][V] = {};
  int turn = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * blockDim.y; row0 < P.rows;
       row0 += static_cast<int64_t>(gridDim.x) * blockDim.y, turn ^= 1) {
    const int64_t row = row0 + threadIdx.y;
    const bool live = row < P.rows;
    const T* h = static_cast<const T*>(P.h) + row * P.hs;
    const T* gy = static_cast<const T*>(P.gy) + row * P.gys;
    const T* gh = static_cast<const T*>(P.gh) + row * P.ghs;
    T* gx = static_cast<T*>(P.gx) + row * P.gxs;
    Pack<T, V> a[NV], b[NV], c[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool on = live && U::col(j) < P.width;
      a[j] = load_unit<T, V>(h, U::col(j), on);
      b[j] = load_unit<T, V>(gy, U::col(j), on);
    }
    if (P.gh) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        c[j] = load_unit<T, V>(gh, U::col(j), live && U::col(j) < P.width);
    }
    float sum[2] = {0.f, 0.f};  // squares of h; d times h
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V], g[V], w[V];
      unit_floats<T, V>(a[j], f);
      unit_floats<T, V>(b[j], g);
      load_weight<T, V>(P.weight, P.w32, U::col(j), U::col(j) < P.width, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sum[0] = fmaf(f[i], f[i], sum[0]);
        sum[1] = fmaf(g[i] * w[i], f[i], sum[1]);
      }
    }
    row_sums(sum, parts[turn]);
    const float width = static_cast<float>(P.width);
    const float u = rsqrtf(__fdiv_rn(sum[0], width) + P.eps);
    const float mean = __fdiv_rn(sum[1] * u, width);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = U::col(j);
      if (!live || col >= P.width) continue;
      float f[V], g[V], w[V], r[V] = {};
      unit_floats<T, V>(a[j], f);
      unit_floats<T, V>(b[j], g);
      load_weight<T, V>(P.weight, P.w32, col, true, w);
      if (P.gh) unit_floats<T, V>(c[j], r);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float unit = f[i] * u;
        acc[j][i] = fmaf(g[i], unit, acc[j][i]);
        r[i] = fmaf(u, g[i] * w[i] - unit * mean, r[i]);
      }
      store_unit<T, V>(gx, col, unit_of<T, V>(r));
    }
  }
  if (!P.partial) return;
  float* to = P.partial + (static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y) * P.width;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (U::col(j) < P.width) to[U::col(j) + i] = acc[j][i];
}

// Sums of the columns of [parts][width], 32 columns a CTA: every segment of the
// threads sums each 32nd part, then the segments are added in their order.
__global__ void __launch_bounds__(32 * kSumSegments)
    column_sums_kernel(const float* __restrict__ partial, int parts, int width,
                       float* __restrict__ out) {
  __shared__ float sums[kSumSegments][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (col < width) {
#pragma unroll 8
    for (int p = threadIdx.y; p < parts; p += kSumSegments)
      s += partial[static_cast<int64_t>(p) * width + col];
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y || col >= width) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumSegments; ++i) s += sums[i][threadIdx.x];
  out[col] = s;
}

tbe_status check_norm(int32_t dtype, const void* weight, int32_t weight_dtype, int64_t rows,
                      int64_t width, float eps) {
  if (rows < 0 || width < 1 || !(eps >= 0.f) || !(eps < INFINITY)) return TBE_EINVAL;
  if (!dtype_bytes(dtype)) return TBE_EUNSUPPORTED;
  if (weight && weight_dtype != dtype && weight_dtype != TBE_DT_F32) return TBE_EUNSUPPORTED;
  if (weight && !aligned_to(weight, dtype_bytes(weight_dtype))) return TBE_EINVAL;
  if (rows > INT32_MAX || width > TBE_MAX_NORM_WIDTH) return TBE_EUNSUPPORTED;
  return TBE_OK;
}

struct Shape {
  int threads, units, rows;  // of a row, of a thread, of a CTA
};

// How a row is shared: `units` vectors or elements a row, `least` to `most` of them a thread.
Shape shape_of(int64_t rows, int64_t units, int least, int most, int wanted) {
  int threads = 32;
  while (threads < kNormThreads && threads * wanted < units) threads *= 2;
  int per = least;
  while (per * threads < units && per < most) per *= 2;
  Shape s = {threads, per, 1};
  while (s.rows * s.threads < kNormCta && s.rows * 152 * 4 < rows) s.rows *= 2;
  return s;
}

// Calls f with the number of units of a thread as a constant.
template <int kLeast, typename F>
void for_units(int units, F f) {
  if (units == kLeast) f(std::integral_constant<int, kLeast>{});
  else if (units == kLeast * 2) f(std::integral_constant<int, kLeast * 2>{});
  else if (units == kLeast * 4) f(std::integral_constant<int, kLeast * 4>{});
  else f(std::integral_constant<int, kLeast * 8>{});
}

template <bool kFp8>
tbe_status run_norm(const void* x, const void* residual, const void* weight, int32_t dtype,
                    int32_t weight_dtype, int64_t rows, int64_t width, int64_t x_stride,
                    int64_t residual_stride, float eps, void* h, int64_t h_stride, void* y,
                    int64_t y_stride, float* scale, void* stream) {
  const tbe_status bad = check_norm(dtype, weight, weight_dtype, rows, width, eps);
  if (bad != TBE_OK) return bad;
  if (!rows) return TBE_OK;
  const int b = dtype_bytes(dtype);
  const Matrix in[2] = {{x, x_stride, b}, {residual, residual_stride, b}};
  const Matrix out[2] = {{y, y_stride, kFp8 ? 1 : b}, {h, h_stride, b}};
  if (!in[0].good(rows, width) || !out[0].good(rows, width) ||
      (residual && !in[1].good(rows, width)) || (h && (!residual || !out[1].good(rows, width))) ||
      (kFp8 && (!scale || !aligned_to(scale, 4))))
    return TBE_EINVAL;
  const int64_t blocks = (width + kBlock - 1) / kBlock;
  const Bytes read[3] = {in[0].span(rows, width), in[1].span(rows, width),
                         run_of(weight, weight ? width * dtype_bytes(weight_dtype) : 0)};
  const Bytes written[3] = {out[0].span(rows, width), out[1].span(rows, width),
                            run_of(kFp8 ? scale : nullptr, rows * blocks * 4)};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 3; ++j)
      if (overlap(written[i], read[j]) || (j < i && overlap(written[i], written[j])))
        return TBE_EINVAL;
  const bool vec = in[0].vectors(width, 16) && (!residual || in[1].vectors(width, 16)) &&
                   (!h || out[1].vectors(width, 16)) && aligned_to(weight, 16) &&
                   out[0].vectors(width, kFp8 ? 16 / b : 16);
  const NormArgs args = {x, residual, weight, h, y, scale, x_stride, residual_stride, h_stride,
                         y_stride, static_cast<int>(rows), static_cast<int>(width),
                         weight_dtype == TBE_DT_F32, eps};
  return for_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const auto go = [&](auto aligned, const Shape& s) {
      constexpr bool kAligned = decltype(aligned)::value;
      for_units<kAligned ? 1 : 4>(s.units, [&](auto n) {
        rms_norm_kernel<T, kFp8, kAligned, decltype(n)::value>
            <<<static_cast<unsigned>((rows + s.rows - 1) / s.rows), dim3(s.threads, s.rows), 0,
               static_cast<cudaStream_t>(stream)>>>(args);
      });
      return launched();
    };
    if (vec) return go(std::true_type{}, shape_of(rows, width / kVec<T>, 1, 8, rows < 608 ? 1 : 4));
    return go(std::false_type{}, shape_of(rows, width, 4, 32, 8));
  });
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_rms_norm(const void* x, const void* residual, const void* weight,
                                   int32_t dtype, int32_t weight_dtype, int64_t rows,
                                   int64_t width, int64_t x_stride, int64_t residual_stride,
                                   float eps, void* h, int64_t h_stride, void* y,
                                   int64_t y_stride, void* stream) {
  return run_norm<false>(x, residual, weight, dtype, weight_dtype, rows, width, x_stride,
                         residual_stride, eps, h, h_stride, y, y_stride, nullptr, stream);
}

extern "C" tbe_status tbe_rms_norm_fp8(const void* x, const void* residual, const void* weight,
                                       int32_t dtype, int32_t weight_dtype, int64_t rows,
                                       int64_t width, int64_t x_stride, int64_t residual_stride,
                                       float eps, void* h, int64_t h_stride, uint8_t* q,
                                       int64_t q_stride, float* scale, void* stream) {
  return run_norm<true>(x, residual, weight, dtype, weight_dtype, rows, width, x_stride,
                        residual_stride, eps, h, h_stride, q, q_stride, scale, stream);
}

extern "C" tbe_status tbe_rms_norm_workspace_size(int64_t rows, int64_t width, size_t* bytes) {
  if (rows < 0 || width < 1 || !bytes) return TBE_EINVAL;
  if (rows > INT32_MAX || width > TBE_MAX_NORM_WIDTH) return TBE_EUNSUPPORTED;
  *bytes = static_cast<size_t>(rows < kNormParts ? rows : kNormParts) * width * 4;
  return TBE_OK;
}

extern "C" tbe_status tbe_rms_norm_backward(const void* grad_y, const void* h, const void* weight,
                                            const void* grad_h, int32_t dtype,
                                            int32_t weight_dtype, int64_t rows, int64_t width,
                                            int64_t grad_y_stride, int64_t h_stride,
                                            int64_t grad_h_stride, float eps, void* grad_x,
                                            int64_t grad_x_stride, float* grad_weight,
                                            void* workspace, size_t ws_bytes, void* stream) {
  const tbe_status bad = check_norm(dtype, weight, weight_dtype, rows, width, eps);
  if (bad != TBE_OK) return bad;
  if (!aligned_to(grad_weight, 4)) return TBE_EINVAL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int b = dtype_bytes(dtype);
  const Matrix in[3] = {{grad_y, grad_y_stride, b}, {h, h_stride, b}, {grad_h, grad_h_stride, b}};
  const Matrix out = {grad_x, grad_x_stride, b};
  size_t need = 0;
  if (rows) {
    if (!in[0].good(rows, width) || !in[1].good(rows, width) ||
        (grad_h && !in[2].good(rows, width)) || !out.good(rows, width))
      return TBE_EINVAL;
    if (grad_weight) {
      tbe_rms_norm_workspace_size(rows, width, &need);
      if (!workspace || ws_bytes < need || !aligned_to(workspace, 16)) return TBE_EWORKSPACE;
    }
  }
  const Bytes read[4] = {in[0].span(rows, width), in[1].span(rows, width),
                         in[2].span(rows, width),
                         run_of(weight, weight ? width * dtype_bytes(weight_dtype) : 0)};
  const Bytes written[3] = {out.span(rows, width), run_of(grad_weight, width * 4),
                            run_of(need ? workspace : nullptr, static_cast<int64_t>(need))};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 4; ++j)
      if (overlap(written[i], read[j])) return TBE_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return TBE_EINVAL;
  }
  int parts = 0;
  if (rows) {
    const bool vec = in[0].vectors(width, 16) && in[1].vectors(width, 16) &&
                     (!grad_h || in[2].vectors(width, 16)) && out.vectors(width, 16) &&
                     aligned_to(weight, 16);
    NormGradArgs args = {grad_y, h, weight, grad_h, grad_x,
                         grad_weight ? static_cast<float*>(workspace) : nullptr,
                         grad_y_stride, h_stride, grad_h_stride, grad_x_stride,
                         static_cast<int>(rows), static_cast<int>(width),
                         weight_dtype == TBE_DT_F32, eps};
    const tbe_status st = for_dtype(dtype, [&](auto t) {
      using T = decltype(t);
      const auto go = [&](auto aligned, Shape sh) {
        constexpr bool kAligned = decltype(aligned)::value;
        while (sh.rows > rows) sh.rows /= 2;
        const int64_t groups = rows / sh.rows, most = kNormParts / sh.rows;
        const int ctas = static_cast<int>(groups < most ? groups : most);
        parts = ctas * sh.rows;
        for_units<kAligned ? 1 : 4>(sh.units, [&](auto n) {
          rms_norm_backward_kernel<T, kAligned, decltype(n)::value>
              <<<ctas, dim3(sh.threads, sh.rows), 0, s>>>(args);
        });
        return launched();
      };
      if (vec) return go(std::true_type{}, shape_of(rows, width / kVec<T>, 1, 8, 1));
      return go(std::false_type{}, shape_of(rows, width, 4, 32, 4));
    });
    if (st != TBE_OK) return st;
  }
  if (!grad_weight) return TBE_OK;
  column_sums_kernel<<<static_cast<unsigned>((width + 31) / 32), dim3(32, kSumSegments), 0, s>>>(
      static_cast<const float*>(workspace), parts, static_cast<int>(width), grad_weight);
  return launched();
}
