// Values to e4m3 with a scale for each block of 128: the arithmetic that
// include/tbe_experts.h specifies at tbe_quantize_weights.
#pragma once

#include <cuda_fp8.h>

#include "rows.cuh"
#include "tbe_experts.h"

namespace tbe {

constexpr int kBlock = TBE_SCALE_BLOCK;
constexpr float kInvMax = 1.f / 448.f;  // one over the largest e4m3 value, rounded to fp32
constexpr float kTinyScale = 0x1p-126f;

__device__ __forceinline__ float block_scale(float amax) {
  return fmaxf(amax * kInvMax, kTinyScale);
}

// Four or eight values times f, to e4m3.
template <int N>
__device__ __forceinline__ Pack<uint8_t, N> to_e4m3(const float (&v)[N], float f) {
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * f, v[4 * i + 1] * f),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * f, v[4 * i + 3] * f),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  Pack<uint8_t, N> p;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) reinterpret_cast<uint32_t*>(&p)[i] = w[i];
  return p;
}

// e4m3(x / s) of four or eight values, as a division in fp32 gives it.  The quotient lies
// between x times a little less and a little more than 1 / s (2^-21 of it is more than
// the errors on the way add up to: 2^-23 of the approximate reciprocal and three
// roundings of 2^-24), and rounding is monotonic, so where both give the same e4m3
// values the quotients do too.  Where they differ (one lane in some thousands) the values
// are divided.  (8192 x 1024 bf16 to four places: 15.0 us, with divisions throughout 17.2.)
template <int N>
__device__ __forceinline__ Pack<uint8_t, N> quantized(const float (&x)[N], float s) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  Pack<uint8_t, N> q = to_e4m3(x, inv * (1.f - 0x1p-21f));
  const Pack<uint8_t, N> more = to_e4m3(x, inv * (1.f + 0x1p-21f));
  bool same = true;
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    same &= reinterpret_cast<const uint32_t*>(&q)[i] == reinterpret_cast<const uint32_t*>(&more)[i];
  if (!same) {
    float d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = __fdiv_rn(x[i], s);
    q = to_e4m3(d, 1.f);
  }
  return q;
}

}  // namespace tbe
