// Root-mean-square norm with the residual's addition, in the rows' type or in
// 8 bits, and its gradients.  The operations are specified in include/tbe_norm.h.
//
// Memory bounds both directions.  A row is shared by 32 to 512 threads, which read it once: its
// squares are summed, and its outputs are formed from registers.  The threads walk rows a grid
// apart, and each copies its own part of the next rows to a ring in shared memory
// (cp.async, private to the thread, so nothing but its own copies is waited for): loads are always
// on their way, whatever the row at hand waits for.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "entry.cuh"
#include "quantize.cuh"
#include "tbe_norm.h"

namespace tbe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kNormThreads = 512;     // threads of a CTA, at most
constexpr int kNormParts = 152 * 8;   // partial sums of grad_weight, at most
constexpr int kNormShared = 220 * 1024;
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
__device__ __forceinline__ Pack<T, V> load_unit(const T* row, int col, bool on) {
  if (on) return *reinterpret_cast<const Pack<T, V>*>(row + col);
  Pack<T, V> zero;
#pragma unroll
  for (int i = 0; i < V; ++i) zero.v[i] = from_f32<T>(0.f);
  return zero;
}
template <typename T, int V>
__device__ __forceinline__ void store_unit(T* row, int col, const Pack<T, V>& p) {
  *reinterpret_cast<Pack<T, V>*>(row + col) = p;
}

// A thread's values are computed on two at a time (one instruction for two multiplications or
// additions): pair i of its units, two neighbours in a vector, or two single elements.
template <typename T, int V, int NV>
__device__ __forceinline__ float2 pair_at(const Pack<T, V> (&p)[NV], int i) {
  if constexpr (V == 1) {
    return make_float2(to_f32(p[2 * i].v[0]), to_f32(p[2 * i + 1].v[0]));
  } else if constexpr (sizeof(T) == 4) {
    const Pack<T, V>& u = p[i / (V / 2)];
    return make_float2(u.v[i % (V / 2) * 2], u.v[i % (V / 2) * 2 + 1]);
  } else {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&p[i / (V / 2)])[i % (V / 2)];
    if constexpr (std::is_same_v<T, __half>)
      return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else  // a bf16 is the upper half of an fp32
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}
template <typename T, int V, int NV>
__device__ __forceinline__ void set_pair(Pack<T, V> (&p)[NV], int i, float2 f) {
  if constexpr (V == 1) {
    p[2 * i].v[0] = from_f32<T>(f.x);
    p[2 * i + 1].v[0] = from_f32<T>(f.y);
  } else if constexpr (sizeof(T) == 4) {
    Pack<T, V>& u = p[i / (V / 2)];
    u.v[i % (V / 2) * 2] = f.x;
    u.v[i % (V / 2) * 2 + 1] = f.y;
  } else {
    uint32_t& w = reinterpret_cast<uint32_t*>(&p[i / (V / 2)])[i % (V / 2)];
    if constexpr (std::is_same_v<T, __half>) {
      const __half2 h = __floats2half2_rn(f.x, f.y);
      w = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      w = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }

// The thread's part of the weight.  In the rows' type it stays in registers; in fp32 beside
// 16-bit rows it is read for each row.
template <typename T, bool kAligned, int NV, bool kShifted>
struct Weight {
  using U = Units<T, kAligned>;
  static constexpr int V = U::V;
  Pack<T, V> own[NV];
  const float* wide;
  int width, lead;

  // lead: columns of the first unit before the row (kShifted).
  __device__ __forceinline__ Weight(const void* weight, bool w32, int width_, int lead_)
      : width(width_), lead(lead_) {
    wide = sizeof(T) == 2 && weight && w32 ? static_cast<const float*>(weight) : nullptr;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (kShifted) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = U::col(j) + i - lead;
          own[j].v[i] = weight && !wide && c >= 0 && c < width ? static_cast<const T*>(weight)[c]
                                                              : from_f32<T>(1.f);
        }
        continue;
      }
      const bool on = weight && !wide && U::col(j) < width;
      own[j] = load_unit<T, V>(static_cast<const T*>(weight), U::col(j), on);
      if (!on)
#pragma unroll
        for (int i = 0; i < V; ++i) own[j].v[i] = from_f32<T>(1.f);
    }
  }
  __device__ __forceinline__ float2 at(int i) const {
    if constexpr (sizeof(T) == 2) {
      if (wide) {
        if constexpr (V == 1) {
          const int a = U::col(2 * i), b = U::col(2 * i + 1);
          return make_float2(a < width ? wide[a] : 1.f, b < width ? wide[b] : 1.f);
        } else {
          const int col = U::col(i / (V / 2)) + i % (V / 2) * 2 - lead;
          if constexpr (kShifted)
            return make_float2(col >= 0 && col < width ? wide[col] : 1.f,
                               col + 1 >= 0 && col + 1 < width ? wide[col + 1] : 1.f);
          return col < width ? *reinterpret_cast<const float2*>(wide + col) : both(1.f);
        }
      }
    }
    return pair_at(own, i);
  }
};

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

// Rows of each of kIn matrices on their way to this thread, kDeep of them a matrix.  (Two vectors a
// thread: two rows ahead; gradients of 65536 x 2048 bf16 156 us, with three 164, four 177.)
template <typename T, bool kAligned, int NV, int kIn>
struct Ahead {
  using U = Units<T, kAligned>;
  static constexpr int kDeep = NV == 1 ? 4 : NV <= 4 ? 2 : 1;
  static constexpr int kBytes = kDeep * kIn * NV * 16;  // of shared memory a thread
  uint4* slots;  // this thread's first; the CTA's threads lie side by side

  __device__ __forceinline__ uint4* slot(int stage, int in, int j) const {
    return slots + ((stage * kIn + in) * NV + j) * (blockDim.x * blockDim.y);
  }
  // From the boundary `lead` columns before the row up to column `end` from there.
  __device__ __forceinline__ void start(int stage, int in, const void* matrix, int64_t stride,
                                        int64_t row, int lead, int end) const {
    const T* from = static_cast<const T*>(matrix) + row * stride - lead;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = U::col(j), bytes = col < end ? 16 : 0;  // the rest are zeros
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<unsigned>(
                       __cvta_generic_to_shared(slot(stage, in, j)))),
                   "l"(from + (bytes ? col : 0)), "r"(bytes)
                   : "memory");
    }
  }
  static __device__ __forceinline__ void close() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // All but the last kDeep - 1 groups are there.
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
  }
  __device__ __forceinline__ Pack<T, kVec<T>> unit(int stage, int in, int j) const {
    return *reinterpret_cast<const Pack<T, kVec<T>>*>(slot(stage, in, j));
  }
  __device__ __forceinline__ void read(int stage, int in, Pack<T, kVec<T>> (&v)[NV]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = unit(stage, in, j);
  }
};

extern __shared__ uint4 norm_ring[];

// The rows that a row of threads walks: `first` of its CTA, its own `row`, then `step` on.  Shifted
// rows are off 16 bytes, by as much as others are every kVec rows; a CTA's are alike, so `lead`,
// the columns between the boundary and the row, is the same for all of a thread's
// rows.  Its vectors begin at the boundary: the first and the last of a row hold other columns, which
// are zeros here and not stored.
template <typename T, bool kShifted>
struct Walk {
  int64_t first, row, step;
  int lead, end;  // columns, from the boundary on

  __device__ __forceinline__ Walk(const void* p, int64_t stride, int width) {
    constexpr int kAlike = kShifted ? kVec<T> : 1;
    const int y = blockDim.y, b = blockIdx.x;
    first = b % kAlike + static_cast<int64_t>(b / kAlike) * y * kAlike;
    row = first + static_cast<int64_t>(threadIdx.y) * kAlike;
    step = static_cast<int64_t>(gridDim.x / kAlike) * y * kAlike;
    lead = kShifted ? tbe::lead<T>(static_cast<const T*>(p) + first * stride) : 0;
    end = lead + width;
  }
  __device__ __forceinline__ void next() { first += step, row += step; }
  // Zeros in a vector's columns outside the row.
  __device__ __forceinline__ void mask(Pack<T, kVec<T>>& v, int col) const {
    if (!kShifted || (col >= lead && col + kVec<T> <= end)) return;
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
      if (col + i < lead || col + i >= end) v.v[i] = from_f32<T>(0.f);
  }
  // `boundary`: the row's start less `lead`.
  __device__ __forceinline__ void store(T* boundary, int col, const Pack<T, kVec<T>>& v) const {
    if (!kShifted || (col >= lead && col + kVec<T> <= end)) {
      store_unit<T, kVec<T>>(boundary, col, v);
    } else {
#pragma unroll
      for (int i = 0; i < kVec<T>; ++i)
        if (col + i >= lead && col + i < end) boundary[col + i] = v.v[i];
    }
  }
};

// kIn: 2 with a residual; rows off 16 bytes, which are loaded where they are needed, ask for it.
template <typename T, bool kFp8, bool kAligned, int NV, int kIn, bool kShifted>
__global__ void __launch_bounds__(kNormThreads)
    rms_norm_kernel(const __grid_constant__ NormArgs P) {
  using U = Units<T, kAligned>;
  constexpr int V = U::V, kPairs = NV * V / 2;
  using Ring = Ahead<T, kAligned, NV, kIn>;
  __shared__ float parts[2][kNormThreads / 32][1];
  Walk<T, kShifted> walk(P.x, P.xs, P.width);
  const int lead = walk.lead, end = walk.end;
  const Ring ring = {norm_ring + threadIdx.y * blockDim.x + threadIdx.x};
  const auto start = [&](int stage, int64_t r) {
    if (r < P.rows) {
      ring.start(stage, 0, P.x, P.xs, r, lead, end);
      if (kIn == 2) ring.start(stage, 1, P.residual, P.rs, r, lead, end);
    }
    ring.close();
  };
  if constexpr (kAligned) {
#pragma unroll
    for (int k = 0; k < Ring::kDeep; ++k) start(k, walk.row + k * walk.step);
  }
  const Weight<T, kAligned, NV, kShifted> weight(P.weight, P.w32, P.width, lead);
  int stage = 0, turn = 0;
  // as many rounds for all rows of the CTA
  for (; walk.first < P.rows; walk.next(), turn ^= 1) {
    const int64_t row = walk.row;
    const bool live = row < P.rows;  // the others take part in the barriers
    Pack<T, V> v[NV];                // zeros from `width` on
    if constexpr (kAligned) {
      ring.wait();
      ring.read(stage, 0, v);
    } else {
      const T* x = static_cast<const T*>(P.x) + row * P.xs;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        v[j] = load_unit<T, V>(x, U::col(j), live && U::col(j) < P.width);
    }
    if (kIn == 2 && (kAligned || P.residual)) {
      Pack<T, V> b[NV];
      if constexpr (kAligned) {
        ring.read(stage, 1, b);
      } else {
        const T* r = static_cast<const T*>(P.residual) + row * P.rs;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          b[j] = load_unit<T, V>(r, U::col(j), live && U::col(j) < P.width);
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i)  // the sum as it is held
        set_pair(v, i, __fadd2_rn(pair_at(v, i), pair_at(b, i)));
      if (P.h && live) {
        T* h = static_cast<T*>(P.h) + row * P.hs - lead;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (U::col(j) < end) {
            if constexpr (kAligned) walk.store(h, U::col(j), v[j]);
            else store_unit<T, V>(h, U::col(j), v[j]);
          }
      }
    }
    if constexpr (kShifted) {
#pragma unroll
      for (int j = 0; j < NV; ++j) walk.mask(v[j], U::col(j));
    }
    float2 squares = both(0.f);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) squares = __ffma2_rn(pair_at(v, i), pair_at(v, i), squares);
    float sum[1] = {squares.x + squares.y};
    row_sums(sum, parts[turn]);
    if constexpr (kAligned) {  // all of the row's slots have been read
      start(stage, row + Ring::kDeep * walk.step);
      stage = stage + 1 == Ring::kDeep ? 0 : stage + 1;
    }
    const float2 u = both(rsqrtf(__fdiv_rn(sum[0], static_cast<float>(P.width)) + P.eps));
    if constexpr (!kFp8) {
      T* y = static_cast<T*>(P.y) + row * P.ys - lead;
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        set_pair(v, i, __fmul2_rn(__fmul2_rn(pair_at(v, i), u), weight.at(i)));
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (live && U::col(j) < end) {
          if constexpr (kAligned) walk.store(y, U::col(j), v[j]);
          else store_unit<T, V>(y, U::col(j), v[j]);
        }
    } else {
      constexpr int kUnits = kAligned ? 1 : 4;          // units of a thread in a block of 128
      constexpr int kLanes = kAligned ? kBlock / V : 32;  // lanes that share it
      constexpr int kHeld = kUnits * V;                 // values of a thread in it
      uint8_t* q = static_cast<uint8_t*>(P.y) + row * P.ys;
      float* scale = P.scale + row * ((P.width + kBlock - 1) / kBlock);
#pragma unroll
      for (int j = 0; j < NV; j += kUnits) {
        float f[kHeld], amax = 0.f;
#pragma unroll
        for (int k = 0; k < kHeld / 2; ++k) {
          const int i = j * V / 2 + k;
          const float2 y = __fmul2_rn(__fmul2_rn(pair_at(v, i), u), weight.at(i));
          f[2 * k] = y.x;
          f[2 * k + 1] = y.y;
          amax = fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y)));  // passes over NaN
        }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
        const float s = block_scale(amax);
        const auto e = quantized(f, s);
        const int col = U::col(j);
        const int first_col = col - (threadIdx.x % kLanes) * V;  // of the block
        if (!live || first_col >= P.width) continue;
        if constexpr (kAligned) {
          if (col < P.width) *reinterpret_cast<Pack<uint8_t, V>*>(q + col) = e;
        } else {
#pragma unroll
          for (int k = 0; k < kUnits; ++k)
            if (U::col(j + k) < P.width) q[U::col(j + k)] = e.v[k];
        }
        if (threadIdx.x % kLanes == 0) scale[first_col / kBlock] = s;
      }
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

// Each thread keeps its columns' part of grad_weight in registers, and its part of the row
// too, unless that is so much that registers run out: then both passes over it read the ring
// (65536 x 2048 bf16 shared by 64 threads: 222 us, with the row in registers 285).  kIn: 3 with a
// gradient that arrives at h.
template <typename T, bool kAligned, int NV, int kIn, bool kShifted>
__global__ void __launch_bounds__(kNormThreads)
    rms_norm_backward_kernel(const __grid_constant__ NormGradArgs P) {
  using U = Units<T, kAligned>;
  constexpr int V = U::V, kPairs = NV * V / 2;
  constexpr int kStep = V == 1 ? 2 : 1, kIn1 = kStep * V / 2;  // units taken at once, their pairs
  constexpr bool kHold = !kAligned || kPairs < 16;
  using Ring = Ahead<T, kAligned, NV, kIn>;
  __shared__ float parts[2][kNormThreads / 32][2];
  float2 acc[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) acc[i] = both(0.f);
  Walk<T, kShifted> walk(P.h, P.hs, P.width);
  const int lead = walk.lead, end = walk.end;
  const Ring ring = {norm_ring + threadIdx.y * blockDim.x + threadIdx.x};
  const auto start = [&](int stage, int64_t r) {
    if (r < P.rows) {
      ring.start(stage, 0, P.h, P.hs, r, lead, end);
      ring.start(stage, 1, P.gy, P.gys, r, lead, end);
      if (kIn == 3) ring.start(stage, 2, P.gh, P.ghs, r, lead, end);
    }
    ring.close();
  };
  if constexpr (kAligned) {
#pragma unroll
    for (int k = 0; k < Ring::kDeep; ++k) start(k, walk.row + k * walk.step);
  }
  const Weight<T, kAligned, NV, kShifted> weight(P.weight, P.w32, P.width, lead);
  int stage = 0, turn = 0;
  for (; walk.first < P.rows; walk.next(), turn ^= 1) {
    const int64_t row = walk.row, step = walk.step;
    const bool live = row < P.rows;
    const T* from[3] = {static_cast<const T*>(P.h) + row * P.hs,
                        static_cast<const T*>(P.gy) + row * P.gys,
                        P.gh ? static_cast<const T*>(P.gh) + row * P.ghs : nullptr};
    if constexpr (kAligned) ring.wait();
    Pack<T, V> held[kIn][kHold ? NV : 1];
    if constexpr (kHold) {
#pragma unroll
      for (int in = 0; in < kIn; ++in)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if constexpr (kAligned) held[in][j] = ring.unit(stage, in, j);
          if constexpr (kShifted) walk.mask(held[in][j], U::col(j));
          if constexpr (!kAligned)
            held[in][j] = load_unit<T, V>(from[in], U::col(j),
                                          live && from[in] && U::col(j) < P.width);
        }
    }
    const auto take = [&](int in, int j, Pack<T, V> (&v)[kStep]) {
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        if constexpr (kHold) v[k] = held[in][j + k];
        else v[k] = ring.unit(stage, in, j + k);
        if constexpr (kShifted && !kHold) walk.mask(v[k], U::col(j + k));
      }
    };
    float2 squares = both(0.f), dots = both(0.f);  // of h; of d and h
#pragma unroll
    for (int j = 0; j < NV; j += kStep) {
      Pack<T, V> a[kStep], b[kStep];
      take(0, j, a);
      take(1, j, b);
#pragma unroll
      for (int i = 0; i < kIn1; ++i) {
        const float2 f = pair_at(a, i);
        squares = __ffma2_rn(f, f, squares);
        dots = __ffma2_rn(__fmul2_rn(pair_at(b, i), weight.at(j * V / 2 + i)), f, dots);
      }
    }
    // what the slots of no row hold must not reach the sums
    float sum[2] = {live ? squares.x + squares.y : 0.f, live ? dots.x + dots.y : 0.f};
    row_sums(sum, parts[turn]);
    const int used = stage;
    if constexpr (kAligned) {
      if (kHold) start(used, row + Ring::kDeep * step);
      if (kHold) stage = stage + 1 == Ring::kDeep ? 0 : stage + 1;
    }
    const float width = static_cast<float>(P.width);
    const float2 u = both(rsqrtf(__fdiv_rn(sum[0], width) + P.eps));
    const float2 mean = both(-__fdiv_rn(sum[1] * u.x, width));
    T* gx = static_cast<T*>(P.gx) + row * P.gxs - lead;
#pragma unroll
    for (int j = 0; j < NV; j += kStep) {
      Pack<T, V> a[kStep], b[kStep], c[kStep];
      take(0, j, a);
      take(1, j, b);
      if constexpr (kIn == 3) take(2, j, c);
#pragma unroll
      for (int i = 0; i < kIn1; ++i) {
        const int at = j * V / 2 + i;
        const float2 unit = __fmul2_rn(pair_at(a, i), u), g = pair_at(b, i);
        if (live) acc[at] = __ffma2_rn(g, unit, acc[at]);
        const float2 d = __ffma2_rn(unit, mean, __fmul2_rn(g, weight.at(at)));
        if constexpr (kIn == 3) set_pair(a, i, __ffma2_rn(u, d, pair_at(c, i)));
        else set_pair(a, i, __fmul2_rn(u, d));
      }
#pragma unroll
      for (int k = 0; k < kStep; ++k)
        if (live && U::col(j + k) < end) {
          if constexpr (kAligned) walk.store(gx, U::col(j + k), a[k]);
          else store_unit<T, V>(gx, U::col(j + k), a[k]);
        }
    }
    if constexpr (kAligned && !kHold) {
      start(used, row + Ring::kDeep * step);
      stage = stage + 1 == Ring::kDeep ? 0 : stage + 1;
    }
  }
  if (!P.partial) return;
  if (blockDim.y > 1) {  // the CTA's groups meet in the ring, which is done with
    float2* sums = reinterpret_cast<float2*>(norm_ring);
    if constexpr (kAligned) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      sums[(i * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x] = acc[i];
    __syncthreads();
    if (threadIdx.y) return;
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      for (int y = 1; y < static_cast<int>(blockDim.y); ++y)
        acc[i] = __fadd2_rn(acc[i], sums[(i * blockDim.y + y) * blockDim.x + threadIdx.x]);
  }
  float* to = P.partial + static_cast<int64_t>(blockIdx.x) * P.width;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    if constexpr (V == 1) {
      if (U::col(2 * i) < P.width) to[U::col(2 * i)] = acc[i].x;
      if (U::col(2 * i + 1) < P.width) to[U::col(2 * i + 1)] = acc[i].y;
    } else {
      const int col = U::col(i / (V / 2)) + i % (V / 2) * 2 - lead;
      if constexpr (kShifted) {
        if (col >= 0 && col < P.width) to[col] = acc[i].x;
        if (col + 1 >= 0 && col + 1 < P.width) to[col + 1] = acc[i].y;
      } else if (col < P.width) {
        to[col] = acc[i].x, to[col + 1] = acc[i].y;
      }
    }
  }
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

// Vectors of a thread, at most: TBE_MAX_NORM_WIDTH columns over kNormThreads threads.
template <typename T>
constexpr int kMostUnits = TBE_MAX_NORM_WIDTH / kVec<T> / kNormThreads;

struct Shape {
  int threads, units, rows;  // of a row, of a thread, of a CTA
};

// How a row of `units` vectors or elements is shared: about `wanted` of them a thread, in whole
// warps up to kNormThreads, `least` to `most` in the end; and rows of a CTA, up to `cta` threads
// and while there are several CTAs a multiprocessor.
Shape shape_of(int64_t units, int least, int most, int wanted) {
  const int64_t warps = (units + 32 * wanted - 1) / (32 * wanted);
  const int threads = static_cast<int>(std::min<int64_t>(warps * 32, kNormThreads));
  int per = least;
  while (per * threads < units && per < most) per *= 2;
  return {threads, per, 1};
}
Shape with_rows(Shape s, int64_t rows, int cta) {
  while (2 * s.rows * s.threads <= cta && s.rows * 152 * 4 < rows) s.rows *= 2;
  return s;
}

// Forward: four vectors a thread (65536 x 2048 bf16 with a residual to 8 bits: one 178 us, two 167,
// four 153; 16384 x 8192: two 184, four 159), but one while the rows are few and latency counts.
// Rows of one warp share a CTA of 256 threads; the others' barriers would tie rows to one another
// (153 us with a row a CTA, 160 with four).
Shape forward_shape(int64_t rows, int64_t vectors, int most) {
  const Shape s = shape_of(vectors, 1, most, rows < 152 * 4 ? 1 : 4);
  return with_rows(s, rows, s.threads == 32 ? 256 : s.threads);
}
// Backward: two vectors a thread (65536 x 2048 bf16: one 199 us, two 156, four 222), a CTA a row
// (two rows 159 us, four 165), but of 256 threads for rows of one warp, so that few parts are left
// to add (65536 x 256 bf16: 24.5 us and 3.4 for the parts; a CTA a row 31.0 and 5.2).
Shape backward_shape(int64_t rows, int64_t vectors, int most) {
  const Shape s = shape_of(vectors, 1, most, 2);
  return with_rows(s, rows, s.threads == 32 ? 256 : s.threads);
}

// Whether rows of the matrices are off 16 bytes alike.
bool alike(const Matrix* m, int n) {
  const auto off = [](const Matrix& a, const Matrix& b) {
    const uintptr_t starts = reinterpret_cast<uintptr_t>(a.p) ^ reinterpret_cast<uintptr_t>(b.p);
    return (starts | (static_cast<uint64_t>(a.stride) - static_cast<uint64_t>(b.stride)) *
                         static_cast<uint64_t>(a.bytes)) % 16 != 0;
  };
  for (int i = 1; i < n; ++i)
    if (m[i].p && off(m[i], m[0])) return false;
  return true;
}

// Whether rows off 16 bytes alike are moved in the vectors of their boundaries (Walk), where those fit
// the threads: 65536 x 1001 bf16 44 us and by single elements 114, with a residual 93 and 142, gradients
// 102 and 171.  But up to 128 columns, four elements of a warp's threads, those are faster (100000
// x 101: 18 us, in vectors 23; x 137: 33 and 23), and for the gradients of few rows, as a thread has
// more rows one after another in vectors (300 x 1001: 5.6 us and 6.9, 4000: 16.2 and 15.5).
template <typename T>
bool in_shifted_vectors(int64_t width) {
  return width > 128 && (width + 2 * kVec<T> - 2) / kVec<T> <= kMostUnits<T> * kNormThreads;
}
constexpr int64_t kShiftedGradRows = 152 * 16;

// CTAs of a launch: as many as fit the GPU with `bytes` of shared memory and as many registers a
// thread, or fewer.  alike: they come in so many kinds (Walk).
int64_t ctas_of(const Shape& s, int64_t rows, int bytes, int registers, int alike) {
  const int threads = s.threads * s.rows;
  const int regs = 65536 / ((registers + 7) / 8 * 8) / threads;
  const int fit = std::max(
      1, std::min({regs, 2048 / threads, kNormShared / (bytes * threads + 1024), 32}));
  const int64_t each = (rows + alike - 1) / alike;  // rows of a kind
  return std::min<int64_t>((each + s.rows - 1) / s.rows * alike, int64_t(152) * fit);
}

template <typename Args>
int registers_of(void (*kernel)(Args)) {
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, kernel) == cudaSuccess) return a.numRegs;
  cudaGetLastError();
  return 128;
}

template <typename Args>
tbe_status launch_norm(void (*kernel)(Args), const Args& args, const Shape& s, int64_t ctas,
                       int bytes, void* stream) {
  const int smem = bytes * s.threads * s.rows;
  // What is asked for is the kernel's and not the launch's: as much for every launch of it, so that
  // none takes from another, which a second host thread may be about to make or a graph holds.
  const int most = bytes * kNormThreads;
  if (most > 40 * 1024 &&  // beside what is declared in the kernels
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) !=
          cudaSuccess)
    return refused();
  kernel<<<static_cast<unsigned>(ctas), dim3(s.threads, s.rows), smem,
           static_cast<cudaStream_t>(stream)>>>(args);
  return launched();
}

template <int N>
using Int = std::integral_constant<int, N>;

// Calls f with the number of units of a thread as a constant.
template <int kLeast, int kMost, typename F>
void for_units(int units, F f) {
  if (units == kLeast) f(Int<kLeast>{});
  else if (units == kLeast * 2) f(Int<kLeast * 2>{});
  else if (units == kLeast * 4 || kMost == kLeast * 4) f(Int<kLeast * 4>{});
  else f(Int<kMost>{});
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
    const auto go = [&](auto aligned, auto shifted, auto in, const Shape& s) {
      constexpr bool kAligned = decltype(aligned)::value, kShifted = decltype(shifted)::value;
      constexpr int kIn = decltype(in)::value;
      tbe_status st = TBE_OK;
      for_units<kAligned ? 1 : 4, kAligned ? kMostUnits<T> : 32>(s.units, [&](auto n) {
        constexpr int NV = decltype(n)::value;
        constexpr int kBytes = kAligned ? Ahead<T, kAligned, NV, kIn>::kBytes : 0;
        const auto kernel = rms_norm_kernel<T, kFp8, kAligned, NV, kIn, kShifted>;
        static const int registers = registers_of(kernel);
        const int64_t ctas = kAligned
                                 ? ctas_of(s, rows, kBytes, registers, kShifted ? kVec<T> : 1)
                                 : (rows + s.rows - 1) / s.rows;
        st = launch_norm(kernel, args, s, ctas, kBytes, stream);
      });
      return st;
    };
    const auto with = [&](auto shifted, auto in) {
      const int64_t vectors = (width + (vec ? 0 : 2 * kVec<T> - 2)) / kVec<T>;
      return go(std::true_type{}, shifted, in, forward_shape(rows, vectors, kMostUnits<T>));
    };
    // (fp32 rows are summed in one order, so that their norm, quantised, is the norm in 8 bits)
    if constexpr (!kFp8 && sizeof(T) == 2) {
      const Matrix moved[4] = {in[0], in[1], out[0], out[1]};
      if (!vec && alike(moved, 4) && in_shifted_vectors<T>(width))
        return residual ? with(std::true_type{}, Int<2>{}) : with(std::true_type{}, Int<1>{});
    }
    if (!vec)
      return go(std::false_type{}, std::false_type{}, Int<2>{},
                with_rows(shape_of(width, 4, 32, 8), rows, 256));
    return residual ? with(std::false_type{}, Int<2>{}) : with(std::false_type{}, Int<1>{});
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
    const NormGradArgs args = {grad_y, h, weight, grad_h, grad_x,
                         grad_weight ? static_cast<float*>(workspace) : nullptr,
                         grad_y_stride, h_stride, grad_h_stride, grad_x_stride,
                         static_cast<int>(rows), static_cast<int>(width),
                         weight_dtype == TBE_DT_F32, eps};
    const tbe_status st = for_dtype(dtype, [&](auto t) {
      using T = decltype(t);
      const auto go = [&](auto aligned, auto shifted, auto in, Shape sh) {
        constexpr bool kAligned = decltype(aligned)::value, kShifted = decltype(shifted)::value;
        constexpr int kIn = decltype(in)::value, kAlike = kShifted ? kVec<T> : 1;
        while (sh.rows > 1 && sh.rows * kAlike > rows) sh.rows /= 2;
        tbe_status st = TBE_OK;
        for_units<kAligned ? 1 : 4, kAligned ? kMostUnits<T> : 32>(sh.units, [&](auto n) {
          constexpr int NV = decltype(n)::value;
          // a ring, or room for the groups' sums; the ring has room for them
          constexpr int kSums = NV * Units<T, kAligned>::V * 4;
          constexpr int kBytes = kAligned ? Ahead<T, kAligned, NV, kIn>::kBytes : kSums;
          static_assert(kBytes >= kSums, "");
          // whole groups of rows only, so that the parts are no more than the rows
          const auto kernel = rms_norm_backward_kernel<T, kAligned, NV, kIn, kShifted>;
          static const int registers = registers_of(kernel);
          const int64_t ctas = std::min({ctas_of(sh, rows, kBytes, registers, kAlike),
                                         rows / (sh.rows * kAlike) * kAlike, int64_t(kNormParts)});
          parts = static_cast<int>(ctas);
          st = launch_norm(kernel, args, sh, ctas, kBytes, s);
        });
        return st;
      };
      const auto with = [&](auto shifted, auto in) {
        const int64_t vectors = (width + (vec ? 0 : 2 * kVec<T> - 2)) / kVec<T>;
        return go(std::true_type{}, shifted, in, backward_shape(rows, vectors, kMostUnits<T>));
      };
      const Matrix moved[4] = {in[0], in[1], in[2], out};
      if (!vec && rows >= kShiftedGradRows && alike(moved, 4) && in_shifted_vectors<T>(width))
        return grad_h ? with(std::true_type{}, Int<3>{}) : with(std::true_type{}, Int<2>{});
      if (!vec)
        return go(std::false_type{}, std::false_type{}, Int<3>{},
                  with_rows(shape_of(width, 4, 32, 4), rows, 256));
      return grad_h ? with(std::false_type{}, Int<3>{}) : with(std::false_type{}, Int<2>{});
    });
    if (st != TBE_OK) return st;
  }
  if (!grad_weight) return TBE_OK;
  column_sums_kernel<<<static_cast<unsigned>((width + 31) / 32), dim3(32, kSumSegments), 0, s>>>(
      static_cast<const float*>(workspace), parts, static_cast<int>(width), grad_weight);
  return launched();
}
