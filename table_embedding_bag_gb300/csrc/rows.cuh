// Row elements of the expert-layer and gradient kernels: fp32, fp16 or bf16
// values moved in vectors and computed on in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <numeric>
#include <type_traits>

#include "tbe.h"

namespace tbe {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// The one rounding of a result to its type (nearest even).
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// V elements moved by one access (V * sizeof(T) is 16, or V = 1).
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  T v[V];
};

template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// A vector's values in fp32, and the rounding back.
template <typename T>
__device__ __forceinline__ void to_floats(const Pack<T, kVec<T>>& v, float (&f)[kVec<T>]) {
  const uint4 q = *reinterpret_cast<const uint4*>(&v);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same_v<T, __half>) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    } else {  // a bf16 is the upper half of an fp32
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ Pack<T, kVec<T>> from_floats(const float (&f)[kVec<T>]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(f[i]);
    } else if constexpr (std::is_same_v<T, __half>) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  const uint4 q = make_uint4(w[0], w[1], w[2], w[3]);
  return *reinterpret_cast<const Pack<T, kVec<T>>*>(&q);
}

// Elements of T between the 16-byte boundary at or before p and p.
template <typename T>
__device__ __forceinline__ int lead(const void* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
}

// The elements [lo, hi) of a row of `width` that are moved in 16-byte vectors, on
// the 16-byte boundaries of the row `to` that is written; the others, a few at both
// ends, are moved one by one.  kAligned: every row begins on a boundary and ends
// with a whole vector.  Otherwise the inner part leaves out so much that the
// aligned vectors around it lie within the row of any other alignment too.
struct Span {
  int lo, hi;
};
template <typename T, bool kAligned>
__device__ __forceinline__ Span inner_span(const T* to, int width) {
  if constexpr (kAligned) return {0, width};
  const int lo = 2 * kVec<T> - lead<T>(to);
  if (lo + 2 * kVec<T> > width) return {width, width};
  return {lo, lo + ((width - 2 * kVec<T> - lo) / kVec<T> + 1) * kVec<T>};
}

// The 16 bytes that begin `bytes` (an even number) into the 32 of a, b, by selection.
__device__ __forceinline__ uint4 cut(uint4 a, uint4 b, int bytes) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = bytes & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = bytes & 4 ? w[i + 1] : w[i];
  const int bits = (bytes & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// The same by a branch, for lanes on one row, whose vectors are all cut at one place.
__device__ __forceinline__ uint4 cut_row(uint4 a, uint4 b, int bytes) {
  const int bits = (bytes & 3) * 8;
  const auto words = [&](uint32_t p, uint32_t q, uint32_t r, uint32_t s, uint32_t t) {
    return make_uint4(__funnelshift_r(p, q, bits), __funnelshift_r(q, r, bits),
                      __funnelshift_r(r, s, bits), __funnelshift_r(s, t, bits));
  };
  switch (bytes >> 2) {
    case 0: return words(a.x, a.y, a.z, a.w, b.x);
    case 1: return words(a.y, a.z, a.w, b.x, b.y);
    case 2: return words(a.z, a.w, b.x, b.y, b.z);
    default: return words(a.w, b.x, b.y, b.z, b.w);
  }
}

// The vector at p, cut out of the two aligned vectors it lies in.  kBranch: cut by a
// branch, which costs fewer instructions but waits for the loads; the gradients of
// combine, which read a row after the other, gain by it (65536 x 1002 bf16, four rows
// each: 244 us instead of 324), combine, which has four rows' loads in flight, does not.
template <typename T, bool kAligned, bool kBranch = false>
__device__ __forceinline__ Pack<T, kVec<T>> load_vec(const T* __restrict__ p) {
  if constexpr (kAligned) {
    return *reinterpret_cast<const Pack<T, kVec<T>>*>(p);
  } else {
    const int shift = lead<T>(p), bytes = shift * static_cast<int>(sizeof(T));
    const uint4* q = reinterpret_cast<const uint4*>(p - shift);
    const uint4 a = q[0], b = q[shift ? 1 : 0];
    const uint4 o = kBranch ? cut_row(a, b, bytes) : cut(a, b, bytes);
    return *reinterpret_cast<const Pack<T, kVec<T>>*>(&o);
  }
}

template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Pack<T, kVec<T>>& v) {
  *reinterpret_cast<Pack<T, kVec<T>>*>(p) = v;
}

// Calls f(e) for this thread's share of the elements outside the span.
template <typename F>
__device__ __forceinline__ void for_ends(Span s, int width, int t, int threads, F f) {
  const int ends = s.lo + width - s.hi;
  for (int i = t; i < ends; i += threads) f(i < s.lo ? i : s.hi + i - s.lo);
}

inline int dtype_bytes(int32_t dtype) {
  return dtype == TBE_DT_F32 ? 4 : dtype == TBE_DT_F16 || dtype == TBE_DT_BF16 ? 2 : 0;
}

inline bool aligned_to(const void* p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// Rows of `width` bytes, `stride` bytes apart.
struct Bytes {
  const void* p;
  int64_t rows, width, stride;
};
inline Bytes run_of(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }

// Whether the two share memory.  Columns of one buffer beside columns of another row-wise do not;
// where the strides differ, column ranges that meet modulo their greatest common divisor count as
// shared.
inline bool overlap(Bytes a, Bytes b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  if (pa + static_cast<uintptr_t>((a.rows - 1) * a.stride + a.width) <= pb ||
      pb + static_cast<uintptr_t>((b.rows - 1) * b.stride + b.width) <= pa)
    return false;
  if (a.rows == 1 && b.rows == 1) return true;
  const uintptr_t step =
      static_cast<uintptr_t>(a.rows == 1   ? b.stride
                             : b.rows == 1 ? a.stride
                                           : std::gcd(a.stride, b.stride));
  // b's columns, counted from the start of a's
  const uintptr_t at = pb >= pa ? (pb - pa) % step : (step - (pa - pb) % step) % step;
  return at < static_cast<uintptr_t>(a.width) || at + static_cast<uintptr_t>(b.width) > step;
}

}  // namespace tbe
