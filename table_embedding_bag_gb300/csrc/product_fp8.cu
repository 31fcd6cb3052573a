// 8-bit rows and weights with a scale for each block of 128, and the experts'
// products on them.  The operations are specified in include/tbe_experts.h.
#include <cuda.h>
#include <type_traits>

#include "internal.h"
#include "product_form.h"
#include "quantize.cuh"
#include "rows.cuh"
#include "tbe_experts.h"
#include "tcgen05.cuh"

namespace tbe {
namespace {

// Rows and columns are counted in 32 bits, and a block or a tile that begins inside a matrix may
// end past it.
constexpr int64_t kMostRows = INT32_MAX - 512;

// Eight consecutive values of a row.
template <typename T>
struct Eight {
  Pack<T, kVec<T>> v[8 / kVec<T>];
  __device__ __forceinline__ void floats(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8 / kVec<T>; ++i) {
      float x[kVec<T>];
      to_floats<T>(v[i], x);
#pragma unroll
      for (int u = 0; u < kVec<T>; ++u) f[i * kVec<T> + u] = x[u];
    }
  }
  // The largest magnitude; passes over NaN.
  __device__ __forceinline__ float amax() const {
    if constexpr (sizeof(T) == 4) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8 / kVec<T>; ++i)
#pragma unroll
        for (int u = 0; u < kVec<T>; ++u) m = fmaxf(m, fabsf(to_f32(v[i].v[u])));
      return m;
    } else {  // two at a time, exactly
      using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
      const T2* p = reinterpret_cast<const T2*>(v);
      const T2 m = __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])),
                           __hmax2(__habs2(p[2]), __habs2(p[3])));
      return fmaxf(fmaxf(to_f32(m.x), to_f32(m.y)), 0.f);
    }
  }
};

// Values col .. col + 7, zeros from `width` on.
template <typename T, bool kAligned>
__device__ __forceinline__ Eight<T> load8(const T* row, int col, int width) {
  Eight<T> e;
#pragma unroll
  for (int i = 0; i < 8 / kVec<T>; ++i) {
    if (kAligned && col < width) {
      e.v[i] = *reinterpret_cast<const Pack<T, kVec<T>>*>(row + col + i * kVec<T>);
    } else {
#pragma unroll
      for (int u = 0; u < kVec<T>; ++u) {
        const int c = col + i * kVec<T> + u;
        e.v[i].v[u] = !kAligned && c < width ? row[c] : from_f32<T>(0.f);
      }
    }
  }
  return e;
}

template <bool kAligned>
__device__ __forceinline__ void store8(uint8_t* row, int col, int width,
                                       const Pack<uint8_t, 8>& e) {
  if (kAligned) {
    if (col < width) *reinterpret_cast<Pack<uint8_t, 8>*>(row + col) = e;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < width) row[col + i] = e.v[i];
  }
}

// Sixteen lanes quantise a token's block of 128 columns, eight columns each; a
// warp walks the token's blocks two at a time.  The row is read once and all its k
// places are written.  8192 x 1024 bf16 to four places of 32768 takes 14.8 us, 3.5 TB/s (fp16
// 14.5, fp32 12.6; rows that were not in the cache 20.9).  Neither memory nor issue is used up
// (16384 x 2048: DRAM 33 %, issue 60 % at 40 % of the warps), and more warps a multiprocessor do
// not help.  kAligned: rows and q rows allow 16- and 8-byte accesses from end to end.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(256)
    dispatch_fp8_kernel(const T* __restrict__ x, int64_t tokens, int k, int width,
                        int64_t x_stride, const int* __restrict__ offsets, int experts,
                        const int* __restrict__ position, uint8_t* __restrict__ q,
                        int64_t q_stride, float* __restrict__ scale) {
  const int64_t token = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (token >= tokens) return;
  const int blocks = (width + kBlock - 1) / kBlock;
  const int lane = threadIdx.x & 31, half = lane >> 4, col_in = (lane & 15) * 8;
  const int64_t all = tokens * k;
  const T* row = x + token * x_stride;
  const int* pos = position + token * k;
  // gridDim.y warps share a token's pairs of blocks; the next pair's values are on their way
  // while one is quantised.  Four places' addresses are formed before the loop.
  constexpr int kPlaces = 4;
  uint8_t* q_to[kPlaces];
  float* scale_to[kPlaces];
#pragma unroll
  for (int j = 0; j < kPlaces; ++j) {
    const int64_t p = j < k ? (position ? pos[j] : token) : -1;
    const bool on = p >= 0 && p < all;
    q_to[j] = on ? q + p * q_stride : nullptr;
    scale_to[j] = on ? scale + p * blocks : nullptr;
  }
  const int step = gridDim.y * 2;
  Eight<T> next = load8<T, kAligned>(row, (blockIdx.y * 2 + half) * kBlock + col_in, width);
  for (int b0 = blockIdx.y * 2; b0 < blocks; b0 += step) {
    const int b = b0 + half;
    const int col = b * kBlock + col_in;
    float in[8];
    next.floats(in);
    float amax = next.amax();
    if (b0 + step < blocks) next = load8<T, kAligned>(row, col + step * kBlock, width);
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = block_scale(amax);
    const Pack<uint8_t, 8> e = quantized(in, s);
    const bool mine = col < width, first = col_in == 0 && b < blocks;
#pragma unroll
    for (int j = 0; j < kPlaces; ++j)
      if (q_to[j]) {
        if (mine) store8<kAligned>(q_to[j], col, width, e);
        if (first) scale_to[j][b] = s;
      }
    for (int j = kPlaces; j < k; ++j) {
      const int64_t p = pos[j];
      if (p < 0 || p >= all) continue;
      if (mine) store8<kAligned>(q + p * q_stride, col, width, e);
      if (first) scale[p * blocks + b] = s;
    }
  }
  if (!position) return;
  int64_t kept = offsets[experts];
  kept = kept < 0 ? 0 : kept > all ? all : kept;
  for (int64_t r = token * k < kept ? kept : token * k; r < (token + 1) * k; ++r) {
    for (int c = (blockIdx.y * 32 + lane) * 8; c < width; c += gridDim.y * 256) {
      if (kAligned) {
        *reinterpret_cast<uint2*>(q + r * q_stride + c) = make_uint2(0, 0);
      } else {
        for (int i = 0; i < 8 && c + i < width; ++i) q[r * q_stride + c + i] = 0;
      }
    }
    for (int b = blockIdx.y * 32 + lane; b < blocks; b += gridDim.y * 32)
      scale[r * blocks + b] = kTinyScale;
  }
}

// One CTA a 128 x 128 block of an expert's weights, read once: a thread holds eight
// columns of eight rows, 16 rows apart.  2^27 weights: fp32 103 us, 6.5 TB/s, memory; bf16 97 and
// fp16 83 for three fifths of the bytes: the work on each value.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(256)
    quantize_weights_kernel(const T* __restrict__ w, int64_t n, int64_t k, int nb, int kb,
                            uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ float warp_max[8];
  const int64_t unit = blockIdx.x;
  const int64_t e = unit / (static_cast<int64_t>(nb) * kb);
  const int64_t row0 = unit / kb % nb * kBlock + threadIdx.x / 16;
  const int col = static_cast<int>(unit % kb * kBlock) + threadIdx.x % 16 * 8;
  const int cols = static_cast<int>(k);
  const T* src = w + (e * n + row0) * k;
  Eight<T> in[8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    in[i] = load8<T, kAligned>(src + i * 16 * k, col, row0 + i * 16 < n ? cols : 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, in[i].amax());
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, warp_max[i]);
  const float s = block_scale(amax);
  uint8_t* dst = q + (e * n + row0) * k;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x[8];
    in[i].floats(x);
    store8<kAligned>(dst + i * 16 * k, col, row0 + i * 16 < n ? cols : 0, quantized(x, s));
  }
  if (threadIdx.x == 0) scale[unit] = s;
}

// ------------------------------------------------------------------- product
//
// out[token, n] = sum over blocks b of 128 columns of (a_scale[token, b] *
// w_scale[n / 128, b]) * P_b[token, n], with P_b the block's product of 8-bit
// values: four tcgen05 MMAs (kind::f8f6f4, 32 columns each) into a
// tensor-memory accumulator.  While the tensor cores form the next products,
// the epilogue warps read P_b, scale it and add it to the tile's sums in their
// registers: a scale differs from block to block, so the sum over blocks cannot
// stay in tensor memory.
//
// What bounds it: shared memory, which gives 128 bytes a clock, MMA operands and
// arriving copies together; and tensor memory, which the epilogue reads while the
// MMAs use most of its bandwidth (alone an epilogue warp's reads run at 800 bytes a
// clock, beside MMAs at 150 to 220; a block of 256 columns has 128 KB).  So tiles
// are as large as tensor memory allows, two accumulators of 256 columns, once
// there are enough tokens.  How CTAs share a tile:
//   kPair   two CTAs form 256 tokens x 256 columns of n: an MMA (cta_group::2) reads
//           both CTAs' shared memory, which holds half of the tokens and half of the
//           weight rows in each: two thirds of the bytes of a lone CTA with
//           128 x 256 (65536 rows, 16 experts, 4096 x 4096: 778 us, and 990 in
//           kAlone's tiles)
//   kAlone  a CTA forms 128 tokens x 128 columns, with four accumulators: for fewer
//           or uneven tiles
//   kSplit  the CTAs of a cluster each form a part of the sum over blocks of one
//           kAlone tile, for few tokens; the parts meet in shared memory and are
//           added in the order of the ranks (nothing in the cache: one row, 4096 x 4096:
//           14.4 us, and 16.4 in one part; 128 rows, 1024 x 8192: 17.0 and 24.1)
//
// Warps: 0 issues the TMA copies, 1 the MMAs; 2 and 3 bring the blocks' scales
// to shared memory ahead of their use (an epilogue warp that waits for its own
// scales costs more than the block: 512 us instead of 587 at 4096 x 2048), and clear
// the rows of no expert; 4..11 are the epilogue: warp w holds tokens 32 (w % 4)
// .. + 31 of its CTA (one a lane) and half w / 8 of the columns.  A tile with few tokens copies
// them 32 rows at a time; the other rows of the MMA hold what the buffer held before and
// reach only results that are not stored.
constexpr int kTileM = 128;
constexpr int kScaleRing = 8;  // blocks whose scales stand in shared memory
constexpr int kProductThreads = 384;
constexpr int kRowBox = 32;
constexpr int kScaleWarps = 2;
constexpr int kEpilogueWarps = 8;
constexpr int kTmemColumns = 512;
constexpr int kMaxStages = 5;
constexpr int kStoreBox = 128;  // bytes of a row of a stored box

template <int kTileN, Share kShare>
struct ProductShape {
  static constexpr int kTileRows = kShare == kPair ? 2 * kTileM : kTileM;
  static constexpr int kWRows = kShare == kPair ? kTileN / 2 : kTileN;  // weight rows of a CTA
  static constexpr int kAccumulators = kTmemColumns / kTileN;
  static constexpr int kStageBytes = (kTileM + kWRows) * kBlock;  // tokens, then weight rows
  static constexpr int kStages = kShare == kPair ? 4 : 5;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kHeld = kTileN / 128;  // boxes of 32 rows a warp's staging holds
  static constexpr int kWarpStaging = kHeld * 32 * kStoreBox;
  static constexpr int kSmem = kRing + kEpilogueWarps * kWarpStaging + 1024;
  static constexpr int kSums = kTileN / 2;        // of an epilogue thread
  static constexpr int kBlocksN = kTileN / kBlock;  // scale blocks of n
  static constexpr int kJoinStride = kTileN + 4;  // split sums meet in the ring: [128][..] floats
};

// Test-only builds (-DTBE_TEST_STUCK_DRAIN=polls): after the wait for the last MMAs another one, on
// an mbarrier that nothing arrives on, so that the MMAs' warp reports a wait that ran out after
// its work is done.  0 (every regular build): no such wait.
#ifndef TBE_TEST_STUCK_DRAIN
#define TBE_TEST_STUCK_DRAIN 0
#endif
// Likewise (-DTBE_TEST_STUCK_COPY=polls): the second CTA of a pair, when it has filled its ring
// once, waits for such an mbarrier and gives up, while the first goes on.
#ifndef TBE_TEST_STUCK_COPY
#define TBE_TEST_STUCK_COPY 0
#endif

struct ProductArgs {
  const float* a_scale;
  const float* w_scale;
  const int* offsets;
  void* out;
  int64_t out_stride;
  int* status;
  int rows, n, k, experts;
  int kb, nb, n_tiles;  // blocks of k and of n, tiles of n
  int row_tiles;        // the most row tiles that the experts can have
  bool tma_out;         // the rows of out allow TMA stores
};

struct ProductShared {
  // full: a stage's copies have landed; done: the MMAs that read it are done, so the stage is
  // free and the block's product stands in its accumulator, and the block's scales are there;
  // taken: the accumulator has been read
  unsigned long long full[kMaxStages], done[kMaxStages], taken[4], drain;
  unsigned long long left;   // the pair's other CTA has told how many blocks it has copied
  unsigned long long stuck;  // nothing arrives (TBE_TEST_STUCK_...)
  uint32_t tmem;
  int dead;
  int other_copied;
  float scale[kScaleRing][2][kTileM];  // [block][128 columns of n][token]
  int warp_sum[kProductThreads / 32];
  int tile0[TBE_MAX_EXPERTS + 1];  // first row tile of each expert
};

__device__ __forceinline__ int group_start(const ProductArgs& P, int e) {
  if (!P.offsets) return e ? P.rows : 0;
  const int v = P.offsets[e];
  return v < 0 ? 0 : v > P.rows ? P.rows : v;
}

// A wait of a role: gives up at the bound, or soon after another role has.
// The whole warp calls it and goes on or gives up as one.
__device__ __forceinline__ bool role_wait(unsigned long long* bar, uint32_t parity,
                                          volatile int* dead, uint32_t limit = kSpinLimit) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  bool got = false;
  for (uint32_t i = 0; i < limit && !got; ++i) {
    got = mbar_try_wait(bar, parity);
    if (i > 64 && !got) {
      if (*dead) break;
      __nanosleep(64);
    }
  }
  if (!got) *dead = 1;
  return __all_sync(0xffffffffu, got);
}

// Both barriers' phases are over, asked without waiting: the two questions'
// latencies overlap.
__device__ __forceinline__ bool both_over(unsigned long long* x, uint32_t px,
                                          unsigned long long* y, uint32_t py) {
  uint32_t over;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(over)
      : "r"(smem_u32(x)), "r"(px), "r"(smem_u32(y)), "r"(py)
      : "memory");
  return __all_sync(0xffffffffu, over);
}

__device__ __forceinline__ bool elected() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Of a pair's barriers that count for both CTAs, the one of rank 0.
template <bool kTwo>
__device__ __forceinline__ uint32_t leader_bar(unsigned long long* bar) {
  uint32_t addr = smem_u32(bar);
  if constexpr (kTwo) asm volatile("mapa.shared::cluster.u32 %0, %0, 0;" : "+r"(addr));
  return addr;
}

// Copies a box into this CTA's memory; its bytes are counted at `bar`.
template <bool kTwo>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  if constexpr (kTwo)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Writes to a variable of the CTA `rank` of the cluster.
__device__ __forceinline__ void store_to_cta(int* p, uint32_t rank, int v) {
  uint32_t addr = smem_u32(p);
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void arrive_at_cta(unsigned long long* bar, uint32_t rank) {
  uint32_t addr = smem_u32(bar);
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
  arrive_at(addr);
}
__device__ __forceinline__ void fence_cluster() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

// Arrives, at this CTA's barrier or at both CTAs', when the MMAs issued so far
// are done.
template <bool kTwo>
__device__ __forceinline__ void commit_to(unsigned long long* bar) {
  if constexpr (kTwo)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    mma_commit(bar);
}

template <bool kTwo>
__device__ __forceinline__ void take_tmem(uint32_t* slot, uint32_t cols) {
  if constexpr (kTwo) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, cols);
  }
}
template <bool kTwo>
__device__ __forceinline__ void give_tmem(uint32_t base, uint32_t cols) {
  if constexpr (kTwo)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
                 : "memory");
  else
    tmem_dealloc(base, cols);
}

// Operand rows of 128 bytes, written by TMA in its 128-byte swizzle: 8-row
// groups 1024 bytes apart (layout type 2 at bit 61).
__device__ __forceinline__ uint64_t swizzled_desc(const void* p) {
  return make_smem_desc(p, 16, 1024) | (2ull << 61);
}

template <bool kTwo>
__device__ __forceinline__ void mma_f8(uint32_t tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  if constexpr (kTwo)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Starts reading 32 columns of this warp's 32 tensor-memory lanes; the values
// are there after tmem_arrived on the same registers.
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Two fp32 multiply-adds in one instruction: acc += v * s on a pair.  Volatile,
// so that they stay where they are written: after the accumulator is handed back.
__device__ __forceinline__ void fma_pair(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
  uint64_t v;
  asm volatile("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 pair_values(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 load_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote)
               : "memory");
  return v;
}

struct ProductTile {
  int expert, row0, rows, n0;  // first row, rows of the tile, first column
};

// Row tiles of all experts before each, in shared memory; the whole CTA.  Sums
// stop at P.row_tiles, which offsets that rise do not pass.
template <int kTileRows>
__device__ __forceinline__ void build_tiles(const ProductArgs& P, ProductShared& S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int carry = 0;
  for (int e0 = 0; e0 < P.experts; e0 += kProductThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    int tiles = 0;
    if (e < P.experts) {
      const int c = group_start(P, e + 1) - group_start(P, e);
      tiles = c > 0 ? min((c + kTileRows - 1) / kTileRows, P.row_tiles) : 0;
    }
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = min(incl + y, P.row_tiles);
    }
    if (lane == 31) S.warp_sum[warp] = incl;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < kProductThreads / 32; ++w) {
      if (w < warp) before = min(before + S.warp_sum[w], P.row_tiles);
      carry = min(carry + S.warp_sum[w], P.row_tiles);
    }
    if (e < P.experts) S.tile0[e + 1] = min(before + incl, P.row_tiles);
    __syncthreads();
  }
  if (threadIdx.x == 0) S.tile0[0] = 0;
}

// Tile t of the walk: experts in order, and in an expert its row tiles first.
template <int kTileN, int kTileRows>
__device__ __forceinline__ ProductTile tile_at(const ProductArgs& P, const ProductShared& S,
                                               int t) {
  int lo = 0, hi = P.experts - 1;
  while (lo < hi) {  // the last expert whose tiles start at or before t
    const int mid = (lo + hi + 1) >> 1;
    if (S.tile0[mid] * P.n_tiles <= t) lo = mid;
    else hi = mid - 1;
  }
  const int m_tiles = S.tile0[lo + 1] - S.tile0[lo];
  const int at = t - S.tile0[lo] * P.n_tiles;
  const int start = group_start(P, lo), end = group_start(P, lo + 1);
  ProductTile T;
  T.expert = lo;
  T.row0 = start + at % m_tiles * kTileRows;
  T.rows = end - T.row0 < kTileRows ? end - T.row0 : kTileRows;
  T.n0 = at / m_tiles * kTileN;
  return T;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Before a warp writes to its staging buffer: the stores that read it are done
// with it.
__device__ __forceinline__ void staging_free() {
  if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

// One 16-byte part of a row of sums, rounded: elements c .. c + 16 / sizeof(T) - 1.
template <typename T, int kPairs>
__device__ __forceinline__ uint4 rounded(const uint64_t (&acc)[kPairs], int c) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      const float2 f = pair_values(acc[c / 2 + i / 2]);
      w[i] = __float_as_uint(i % 2 ? f.y : f.x);
    } else {
      const float2 f = pair_values(acc[c / 2 + i]);
      w[i] = pack2<T>(f.x, f.y);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Part `i` (16 bytes) of row r of a box in the staging buffer: the 128-byte swizzle of
// TMA, in which the lanes' writes (a row each) spread over the banks.
__device__ __forceinline__ uint4* staged(char* staging, int box, int r, int i) {
  return reinterpret_cast<uint4*>(staging + (box * 32 + r) * kStoreBox + ((i ^ (r & 7)) << 4));
}

// Puts columns c0 .. of the warp's sums into the staging buffer, kHeld boxes of 32
// rows x 128 bytes.
template <typename T, int kSums, int kHeld>
__device__ __forceinline__ void stage(char* staging, int c0, const uint64_t (&acc)[kSums / 2]) {
  constexpr int kCols = kStoreBox / static_cast<int>(sizeof(T));
  constexpr int kPart = 16 / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + h * kCols < kSums)
        *staged(staging, h, lane, i) = rounded<T>(acc, c0 + h * kCols + i * kPart);
}

// Stores a warp's 32 whole rows by TMA: the copies run while the warp goes on to the next
// tile.  (Stores from registers held the tile up: 65536 x 4096 x 1024, 305 us instead
// of 264.)  Columns from n on are clipped.
template <typename T, int kSums, int kHeld>
__device__ __forceinline__ void store_boxes(const ProductArgs& P, const CUtensorMap* map,
                                            char* staging, int row0, int col0,
                                            const uint64_t (&acc)[kSums / 2]) {
  constexpr int kCols = kStoreBox / static_cast<int>(sizeof(T));
#pragma unroll
  for (int c0 = 0; c0 < kSums; c0 += kHeld * kCols) {
    staging_free();
    stage<T, kSums, kHeld>(staging, c0, acc);
    fence_proxy_async();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (c0 + h * kCols < kSums && col0 + c0 + h * kCols < P.n)
          asm volatile(
              "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::
                  "l"(map),
              "r"(col0 + c0 + h * kCols), "r"(row0), "r"(smem_u32(staging + h * 32 * kStoreBox))
              : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
}

// Stores up to 32 rows of any alignment: 16-byte parts on the boundaries of the row of
// out, each cut out of the two staged parts it lies in, and the rows' ends element by
// element.  (65536 rows, 16 experts, 4095 x 2048 bf16: 866 us all element by element.)
template <typename T, int kSums, int kHeld>
__device__ __forceinline__ void store_rows(const ProductArgs& P, char* staging, int row0, int rows,
                                           int col0, const uint64_t (&acc)[kSums / 2]) {
  constexpr int kSize = static_cast<int>(sizeof(T));
  constexpr int kCols = kStoreBox / kSize;
  constexpr int kParts = kHeld * kStoreBox / 16;  // of a row of the buffer
  constexpr int kEnd = 16 / kSize;                // elements of an end, at most
  const int lane = threadIdx.x & 31;
  staging_free();
#pragma unroll
  for (int c0 = 0; c0 < kSums; c0 += kHeld * kCols) {
    if (col0 + c0 >= P.n) break;
    stage<T, kSums, kHeld>(staging, c0, acc);
    __syncwarp();
    int cols = P.n - col0 - c0 < kSums - c0 ? P.n - col0 - c0 : kSums - c0;
    const int bytes = (cols < kHeld * kCols ? cols : kHeld * kCols) * kSize;
    char* to = reinterpret_cast<char*>(static_cast<T*>(P.out) +
                                       static_cast<int64_t>(row0) * P.out_stride + col0 + c0);
    const int64_t pitch = P.out_stride * kSize;
    // bytes from a row's start to its first boundary
    const auto head = [](const char* row) {
      return static_cast<int>(-reinterpret_cast<uintptr_t>(row) & 15);
    };
#pragma unroll 4
    for (int i = lane; i < rows * kParts; i += 32) {
      const int r = i / kParts;
      char* row = to + r * pitch;
      const int at = head(row) + i % kParts * 16;  // counted in the row of the buffer
      if (at + 16 > bytes) continue;
      const int k = at >> 4, shift = at & 15;
      uint4 v = *staged(staging, k >> 3, r, k & 7);
      if (shift) v = cut(v, *staged(staging, (k + 1) >> 3, r, (k + 1) & 7), shift);
      *reinterpret_cast<uint4*>(row + at) = v;
    }
    if (!P.tma_out)
      for (int i = lane; i < rows * 2 * kEnd; i += 32) {
        const int r = i / (2 * kEnd), e = i % (2 * kEnd);
        char* row = to + r * pitch;
        const int first = head(row) < bytes ? head(row) : bytes;
        const int last = first + (bytes - first) / 16 * 16;
        const int at = e < kEnd ? e * kSize : last + (e - kEnd) * kSize;
        if (at < (e < kEnd ? first : bytes))
          *reinterpret_cast<T*>(row + at) = *reinterpret_cast<const T*>(
              reinterpret_cast<const char*>(staged(staging, at >> 7, r, (at >> 4) & 7)) +
              (at & 15));
      }
    __syncwarp();
  }
}

// After a wait that gave up: NaN in this CTA's share of its tiles, finished ones among them, so
// that a product that is not whole does not pass for one.  The whole CTA, when no store is in
// flight.
template <typename T, int kTileN, int kTileRows>
__device__ __forceinline__ void mark_lost(const ProductArgs& P, const ProductShared& S, int first,
                                          int tiles, int stride, int rank, int part, int split) {
  const T nan = from_f32<T>(__int_as_float(0x7fffffff));
  const int cols = kTileN / split;
  for (int t = first; t < tiles; t += stride) {
    const ProductTile tile = tile_at<kTileN, kTileRows>(P, S, t);
    const int rows = min(tile.rows - rank * kTileM, kTileM);
    T* out = static_cast<T*>(P.out) +
             (static_cast<int64_t>(tile.row0) + rank * kTileM) * P.out_stride;
    for (int i = threadIdx.x; i < rows * cols; i += kProductThreads) {
      const int c = tile.n0 + part * cols + i % cols;
      if (c < P.n) out[i / cols * P.out_stride + c] = nan;
    }
  }
}

template <typename T, int kTileN, Share kShare>
__global__ void __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap a_map,
                   const __grid_constant__ CUtensorMap a_part_map,
                   const __grid_constant__ CUtensorMap w_map,
                   const __grid_constant__ CUtensorMap out_map,
                   const __grid_constant__ ProductArgs P) {
  using Shape = ProductShape<kTileN, kShare>;
  constexpr bool kTwo = kShare == kPair;
  constexpr int kTileRows = Shape::kTileRows;
  constexpr int kStages = Shape::kStages, kStageBytes = Shape::kStageBytes;
  constexpr int kSums = Shape::kSums, kAccumulators = Shape::kAccumulators;
  constexpr int kBlocksN = Shape::kBlocksN;
  extern __shared__ char product_smem[];
  __shared__ ProductShared S;
  char* ring = reinterpret_cast<char*>(
      (reinterpret_cast<uintptr_t>(product_smem) + 1023) & ~uintptr_t(1023));
  char* staging = ring + Shape::kRing;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* dead = &S.dead;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.done[i], 1 + kScaleWarps);
    }
    for (int i = 0; i < kAccumulators; ++i)
      mbar_init(&S.taken[i], kTwo ? 2 * kEpilogueWarps : kEpilogueWarps);
    mbar_init(&S.drain, 1);
    mbar_init(&S.left, 1);
    mbar_init(&S.stuck, 1);
    S.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) take_tmem<kTwo>(&S.tmem, kTmemColumns);
  // so far nothing that the kernel before this one writes has been read
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  build_tiles<kTileRows>(P, S);
  fence_before_sync();
  __syncthreads();
  if constexpr (kTwo) cluster_sync();  // the other CTA's barriers are there
  fence_after_sync();
  const uint32_t tmem = S.tmem;
  const int tiles = S.tile0[P.experts] * P.n_tiles;
  const int split = kShare == kSplit ? static_cast<int>(cluster_size()) : 1;
  const int part = kShare == kSplit ? static_cast<int>(cluster_rank()) : 0;
  const int rank = kTwo ? static_cast<int>(cluster_rank()) : 0;
  // a cluster's tiles are first, first + stride, ...; with kSplit it has one
  const int first = static_cast<int>(blockIdx.x) / (kTwo ? 2 : split);
  const int stride = kShare == kSplit ? tiles + 1 : static_cast<int>(gridDim.x) / (kTwo ? 2 : 1);
  const int b0 = static_cast<int>(static_cast<int64_t>(P.kb) * part / split);
  const int b1 = static_cast<int>(static_cast<int64_t>(P.kb) * (part + 1) / split);
  // rows of tokens that the CTA of rank r copies for a tile of `rows` rows
  const auto copied = [](int rows, int r) {
    const int mine = (rows - r * kTileM + kRowBox - 1) / kRowBox * kRowBox;
    return mine <= 0 ? 0 : mine >= kTileM ? kTileM : mine;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      int stage = 0, issued = 0, most = INT32_MAX;
      uint32_t parity = 0;
      bool ok = true;
      // Tells the pair's other CTA how many blocks this one has copied, and whether it gave up.
      const auto tell = [&] {
        if (elected()) {
          store_to_cta(&S.other_copied, rank ^ 1, issued);
          if (!ok) store_to_cta(&S.dead, rank ^ 1, 1);
          fence_cluster();
          arrive_at_cta(&S.left, rank ^ 1);
        }
        __syncwarp();
      };
      for (int t = first; t < tiles && issued < most; t += stride) {
        const ProductTile tile = tile_at<kTileN, kTileRows>(P, S, t);
        const int mine = copied(tile.rows, rank);
        const int row0 = tile.row0 + rank * kTileM;
        const int w0 = tile.expert * P.n + tile.n0 + rank * Shape::kWRows;
        const int bytes = (kTwo ? copied(tile.rows, 0) + copied(tile.rows, 1) + kTileN
                                : mine + kTileN) * kBlock;
        for (int b = b0; b < b1; ++b) {
          const bool stuck = TBE_TEST_STUCK_COPY && kTwo && rank == 1 && issued == kStages;
          if (ok && !(stuck ? role_wait(&S.stuck, 0, dead, TBE_TEST_STUCK_COPY)
                            : role_wait(&S.done[stage], parity ^ 1, dead))) {
            ok = false;
            most = issued;
            // Both CTAs' copies of a block count at rank 0's barrier, which can only be waited for
            // if both are issued.  So the CTA that has issued fewer issues the others'
            // counterparts; their stages are free, or the other CTA would not have filled its own.
            if constexpr (kTwo) {
              tell();
              if (__all_sync(0xffffffffu, mbar_wait(&S.left, 0, 2 * kSpinLimit))) {
                fence_cluster();
                most = max(issued, *static_cast<volatile int*>(&S.other_copied));
              }
            }
          }
          if (issued >= most) break;
          char* a = ring + stage * kStageBytes;
          char* w = a + kTileM * kBlock;
          if (elected()) {
            if (rank == 0) mbar_expect_tx(&S.full[stage], bytes);
            const uint32_t bar = leader_bar<kTwo>(&S.full[stage]);
            tma_load<kTwo>(w, &w_map, b * kBlock, w0, bar);
            if (mine == kTileM)
              tma_load<kTwo>(a, &a_map, b * kBlock, row0, bar);
            else
              for (int r = 0; r < mine; r += kRowBox)
                tma_load<kTwo>(a + r * kBlock, &a_part_map, b * kBlock, row0 + r, bar);
          }
          __syncwarp();
          ++issued;
          if (++stage == kStages) stage = 0, parity ^= 1;
        }
      }
      if (kTwo && ok) tell();
      // Whoever has given up: the copies in flight land before the CTA ends (a pair's are counted
      // at rank 0, and the cluster's last barrier follows).
      for (int i = issued > kStages ? issued - kStages : 0; rank == 0 && i < issued; ++i)
        if (!mbar_wait(&S.full[i % kStages], (i / kStages) & 1)) *dead = 1;
      // Rank 0's MMAs arrive at rank 1's barriers too: rank 1 sees the last arrival before it ends.
      // (It may wait for as long as rank 0 takes to give up, and then for the MMAs.)
      if (rank == 1 && !mbar_wait(&S.drain, 0, 2 * kSpinLimit)) *dead = 1;
    } else if (warp == 1 && rank == 0) {  // a pair's MMAs are issued by rank 0
      const uint32_t idesc = make_idesc(0, kTileRows, kTileN);  // e4m3 x e4m3 -> fp32
      const uint64_t a_desc = swizzled_desc(ring), w_desc = swizzled_desc(ring + kTileM * kBlock);
      int stage = 0, slot = 0;
      uint32_t parity = 0, tparity = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        for (int b = b0; b < b1; ++b) {
          if (!both_over(&S.taken[slot], tparity ^ 1, &S.full[stage], parity) &&
              (!role_wait(&S.taken[slot], tparity ^ 1, dead) ||
               !role_wait(&S.full[stage], parity, dead))) {
            ok = false;
            break;
          }
          fence_after_sync();
          const uint64_t at = static_cast<uint64_t>(stage * (kStageBytes >> 4));
          if (elected()) {
#pragma unroll
            for (int i = 0; i < kBlock / 32; ++i)  // 32 columns are 32 bytes: 2 in the address
              mma_f8<kTwo>(tmem + slot * kTileN, a_desc + at + i * 2, w_desc + at + i * 2, idesc,
                           i > 0);
            commit_to<kTwo>(&S.done[stage]);
          }
          __syncwarp();
          if (++stage == kStages) stage = 0, parity ^= 1;
          if (++slot == kAccumulators) slot = 0, tparity ^= 1;
        }
      }
      // Whoever has given up: the MMAs are done before tensor memory is freed.
      if (elected()) commit_to<kTwo>(&S.drain);
      __syncwarp();
      if (!mbar_wait(&S.drain, 0) ||
          (TBE_TEST_STUCK_DRAIN && !mbar_wait(&S.stuck, 0, TBE_TEST_STUCK_DRAIN)))
        *dead = 1;
    } else if (warp >= 2) {
      // A block's scales replace those of the block kScaleRing earlier.  Those have been read
      // when the MMAs of the block kAccumulators earlier are done, for they took its accumulator.
      constexpr int kAhead = 4;  // blocks whose scales are on their way
      int stage = 0, slot = 0, old_stage = 0, since = 0;
      uint32_t old_parity = 0;
      bool ok = true;
      const int r0 = (warp - 2) * 64 + lane, r1 = r0 + 32;  // this lane's two tokens
      for (int t = first; t < tiles && ok; t += stride) {
        const ProductTile tile = tile_at<kTileN, kTileRows>(P, S, t);
        const int rows = tile.rows - rank * kTileM;
        const float* a0 =
            P.a_scale + (static_cast<int64_t>(tile.row0) + rank * kTileM + r0) * P.kb;
        const float* a1 = a0 + static_cast<int64_t>(32) * P.kb;
        const int wb = tile.n0 / kBlock;
        const float* w0 = P.w_scale + (static_cast<int64_t>(tile.expert) * P.nb + wb) * P.kb;
        const bool on0 = r0 < rows, on1 = r1 < rows, two = kBlocksN == 2 && wb + 1 < P.nb;
        const auto at = [&](const float* p, int b, bool on) {
          return on && b < b1 ? __ldg(p + b) : 0.f;
        };
        float sa0[kAhead], sa1[kAhead], sw[kAhead][kBlocksN];
        const auto load = [&](int i, int b) {
          sa0[i] = at(a0, b, on0);
          sa1[i] = at(a1, b, on1);
          sw[i][0] = at(w0, b, true);
          if constexpr (kBlocksN == 2) sw[i][1] = at(w0 + P.kb, b, two);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(i, b0 + i);
        for (int b4 = b0; b4 < b1 && ok; b4 += kAhead) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int b = b4 + i;
            if (b >= b1) break;
            if (since < kAccumulators) {
              ++since;
            } else {
              if (!role_wait(&S.done[old_stage], old_parity, dead)) {
                ok = false;
                break;
              }
              if (++old_stage == kStages) old_stage = 0, old_parity ^= 1;
            }
#pragma unroll
            for (int h = 0; h < kBlocksN; ++h) {
              S.scale[slot][h][r0] = sa0[i] * sw[i][h];
              S.scale[slot][h][r1] = sa1[i] * sw[i][h];
            }
            __syncwarp();
            if (lane == 0) arrive_at(smem_u32(&S.done[stage]));
            slot = (slot + 1) % kScaleRing;
            load(i, b + kAhead);
            if (++stage == kStages) stage = 0;
          }
        }
      }
      // the rows of no expert: before the first one's and past the last one's
      T* out = static_cast<T*>(P.out);
      const int before = group_start(P, 0), past = group_start(P, P.experts);
      for (int64_t i = blockIdx.x; i < before + static_cast<int64_t>(P.rows - past);
           i += gridDim.x) {
        T* row = out + (i < before ? i : past + (i - before)) * P.out_stride;
        if (P.tma_out)
          for (int c = (threadIdx.x - 64) * kVec<T>; c < P.n; c += 64 * kVec<T>)
            *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
        else
          for (int c = threadIdx.x - 64; c < P.n; c += 64) row[c] = from_f32<T>(0.f);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    char* mine = staging + (warp - 4) * Shape::kWarpStaging;
    const uint32_t taddr0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kSums;
    int stage = 0;
    uint32_t parity = 0, count = 0;  // count: blocks so far
    bool ok = true;
    // test-only builds: a first wait that runs out, to take the way out below
    if (TBE_TEST_STUCK_WAIT && first < tiles)
      ok = role_wait(&S.stuck, 0, dead, TBE_TEST_STUCK_WAIT);
    for (int t = first; t < tiles && ok; t += stride) {
      const ProductTile tile = tile_at<kTileN, kTileRows>(P, S, t);
      const int row0 = tile.row0 + rank * kTileM + quarter * 32;
      const int rows = tile.row0 + tile.rows - row0;  // of this warp; none or less: nothing to do
      const int col0 = tile.n0 + half * kSums;
      const bool on = rows > 0 && col0 < P.n;
      uint64_t acc[kSums / 2];
#pragma unroll
      for (int i = 0; i < kSums / 2; ++i) acc[i] = 0;
      for (int b = b0; b < b1; ++b) {
        if (!role_wait(&S.done[stage], parity, dead)) {
          ok = false;
          break;
        }
        fence_after_sync();
        const uint32_t slot = count % kAccumulators;
        const float sc = S.scale[count % kScaleRing][half * kSums / kBlock][quarter * 32 + lane];
        const uint64_t s = pair_of(sc, sc);
        const uint32_t taddr = taddr0 + slot * kTileN;
        uint32_t v[2][32];
        if (on) {
          tmem_read(taddr, v[0]);
          tmem_read(taddr + 32, v[1]);
          if constexpr (kSums == 128) {  // 64 columns are on their way at a time
            tmem_arrived(v[0]);
            tmem_arrived(v[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                fma_pair(acc[h * 16 + i], v[h][2 * i], v[h][2 * i + 1], s);
              tmem_read(taddr + (2 + h) * 32, v[h]);
            }
          }
          tmem_arrived(v[0]);
          tmem_arrived(v[1]);
        }
        // the accumulator is handed back before its last columns are added
        fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_at(leader_bar<kTwo>(&S.taken[slot]));
        if (on) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              fma_pair(acc[kSums / 2 - 32 + h * 16 + i], v[h][2 * i], v[h][2 * i + 1], s);
        }
        if (++stage == kStages) stage = 0, parity ^= 1;
        ++count;
      }
      if constexpr (kShare == kSplit) {
        if (on && ok) {
          float* join = reinterpret_cast<float*>(ring) +
                        (quarter * 32 + lane) * Shape::kJoinStride + half * kSums;
#pragma unroll
          for (int i = 0; i < kSums / 2; i += 2) {
            const float2 f = pair_values(acc[i]), g = pair_values(acc[i + 1]);
            *reinterpret_cast<float4*>(join + 2 * i) = make_float4(f.x, f.y, g.x, g.y);
          }
        }
      } else if (on && ok) {
        if (rows >= 32 && P.tma_out)
          store_boxes<T, kSums, Shape::kHeld>(P, &out_map, mine, row0, col0, acc);
        else
          store_rows<T, kSums, Shape::kHeld>(P, mine, row0, rows < 32 ? rows : 32, col0, acc);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  if constexpr (kShare == kSplit) {
    if (*dead && lane < split) store_to_cta(&S.dead, lane, 1);  // without one part the sum is lost
    cluster_sync();
    if (first < tiles && !S.dead) {
      const ProductTile tile = tile_at<kTileN, kTileRows>(P, S, first);
      const int quads = kTileN / 4 / split;  // of a row, four columns each
      const uint32_t base = smem_u32(ring);
      T* out = static_cast<T*>(P.out);
      for (int i = threadIdx.x; i < tile.rows * quads; i += kProductThreads) {
        const int r = i / quads, c = (part * quads + i % quads) * 4;
        if (tile.n0 + c >= P.n) continue;
        float4 v[kMostSplit];
#pragma unroll
        for (int p = 0; p < kMostSplit; ++p)
          v[p] = p < split ? load_cluster(base + (r * Shape::kJoinStride + c) * 4, p)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < kMostSplit; ++p) {
          sum[0] += v[p].x;
          sum[1] += v[p].y;
          sum[2] += v[p].z;
          sum[3] += v[p].w;
        }
        T* dst = out + (static_cast<int64_t>(tile.row0) + r) * P.out_stride + tile.n0 + c;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (tile.n0 + c + u < P.n) dst[u] = from_f32<T>(sum[u]);
      }
    }
    cluster_sync();
  }
  fence_before_sync();
  __syncthreads();
  if constexpr (kTwo) cluster_sync();  // the other CTA uses this one's barriers and memory no more
  fence_after_sync();
  if (warp == 2) give_tmem<kTwo>(tmem, kTmemColumns);
  if (S.dead) {
    mark_lost<T, kTileN, kTileRows>(P, S, first, tiles, stride, rank, part, split);
    if (threadIdx.x == 0 && P.status) atomicOr(P.status, TBE_ERR_TIMEOUT);
  }
}

// A map of a matrix of 1-, 2- or 4-byte elements, a row every `stride` bytes, for
// 128-byte-swizzled boxes of 128 bytes x box_rows.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

bool make_map(CUtensorMap* map, const void* base, int bytes, int64_t rows, int64_t cols,
              int64_t stride, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / bytes),
                             static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t steps[2] = {1, 1};
  const CUtensorMapDataType type = bytes == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                                : CU_TENSOR_MAP_DATA_TYPE_UINT32;
  return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  if (tokens > INT32_MAX / k || width > INT32_MAX / 2) return TBE_EUNSUPPORTED;
  if (!tokens || !width) return TBE_OK;
  if (position ? (experts < 1 || !offsets || !aligned_to(offsets, 4) || !aligned_to(position, 4))
               : k != 1)
    return TBE_EINVAL;
  if (!x || !q || !scale || x_stride < width || q_stride < width ||
      !aligned_to(x, dtype_bytes(dtype)) || !aligned_to(scale, 4))
    return TBE_EINVAL;
  const int bytes = dtype_bytes(dtype);
  if (overlap({x, tokens, width * bytes, x_stride * bytes}, {q, tokens * k, width, q_stride}))
    return TBE_EINVAL;
  const bool aligned = width % 8 == 0 && x_stride * bytes % 16 == 0 && q_stride % 8 == 0 &&
                       aligned_to(x, 16) && aligned_to(q, 8);
  // one warp a token once there are enough of them, several for each before
  const int64_t pairs = (width + 2 * kBlock - 1) / (2 * kBlock);
  int64_t share = 152 * 32 / tokens;
  share = share < 1 ? 1 : share > pairs ? pairs : share;
  const dim3 grid(static_cast<unsigned>((tokens + 7) / 8),
                  static_cast<unsigned>(share < 65535 ? share : 65535));
  return for_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const auto kernel = aligned ? dispatch_fp8_kernel<T, true> : dispatch_fp8_kernel<T, false>;
    kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(x), tokens, k, static_cast<int>(width), x_stride, offsets, experts,
        position, q, q_stride, scale);
    return launched();
  });
}

extern "C" tbe_status tbe_quantize_weights(const void* w, int32_t dtype, int64_t experts,
                                           int64_t n, int64_t k, uint8_t* q, float* scale,
                                           void* stream) {
  if (experts < 0 || n < 0 || k < 0) return TBE_EINVAL;
  if (!dtype_bytes(dtype)) return TBE_EUNSUPPORTED;
  if (n > kMostRows || k > kMostRows || experts > INT32_MAX) return TBE_EUNSUPPORTED;
  if (!experts || !n || !k) return TBE_OK;
  if (!w || !q || !scale || !aligned_to(w, dtype_bytes(dtype)) || !aligned_to(scale, 4))
    return TBE_EINVAL;
  const int64_t nb = (n + kBlock - 1) / kBlock, kb = (k + kBlock - 1) / kBlock;
  if (nb * kb > INT32_MAX / experts) return TBE_EUNSUPPORTED;
  if (overlap(run_of(w, experts * n * k * dtype_bytes(dtype)), run_of(q, experts * n * k)))
    return TBE_EINVAL;
  return for_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const bool aligned = k % 8 == 0 && aligned_to(w, 16) && aligned_to(q, 8);
    const auto kernel =
        aligned ? quantize_weights_kernel<T, true> : quantize_weights_kernel<T, false>;
    kernel<<<static_cast<unsigned>(experts * nb * kb), 256, 0,
             static_cast<cudaStream_t>(stream)>>>(static_cast<const T*>(w), n, k,
                                                  static_cast<int>(nb), static_cast<int>(kb), q,
                                                  scale);
    return launched();
  });
}

extern "C" tbe_status tbe_expert_product(const uint8_t* a, int64_t a_stride, const float* a_scale,
                                         const uint8_t* w, const float* w_scale,
                                         const int32_t* offsets, int64_t rows, int64_t n,
                                         int64_t k, int32_t experts, void* out, int32_t out_dtype,
                                         int64_t out_stride, int32_t* status, void* stream) {
  if (rows < 0 || n < 0 || k < 1 || experts < 1) return TBE_EINVAL;
  if (!dtype_bytes(out_dtype)) return TBE_EUNSUPPORTED;
  if (rows > kMostRows || n > kMostRows || k > kMostRows || experts > TBE_MAX_EXPERTS ||
      experts * n > kMostRows)
    return TBE_EUNSUPPORTED;
  if (!rows || !n) return TBE_OK;
  if (!a || !a_scale || !w || !w_scale || !out || (!offsets && experts != 1) || a_stride < k ||
      out_stride < n)
    return TBE_EINVAL;
  if (!aligned_to(a_scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(offsets, 4) ||
      !aligned_to(out, dtype_bytes(out_dtype)) || !aligned_to(status, 4))
    return TBE_EINVAL;
  if (k % 16 || a_stride % 16 || !aligned_to(a, 16) || !aligned_to(w, 16)) return TBE_EUNSUPPORTED;
  const int ob = dtype_bytes(out_dtype);
  const Bytes result = {out, rows, n * ob, out_stride * ob};
  if (overlap({a, rows, k, a_stride}, result) || overlap(run_of(w, experts * n * k), result))
    return TBE_EINVAL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return refused();
  ProductArgs P;
  P.a_scale = a_scale;
  P.w_scale = w_scale;
  P.offsets = offsets;
  P.out = out;
  P.out_stride = out_stride;
  P.status = status;
  P.rows = static_cast<int>(rows);
  P.n = static_cast<int>(n);
  P.k = static_cast<int>(k);
  P.experts = experts;
  P.kb = static_cast<int>((k + kBlock - 1) / kBlock);
  P.nb = static_cast<int>((n + kBlock - 1) / kBlock);
  // (a TMA store clips a row at a multiple of 16 bytes)
  P.tma_out = aligned_to(out, 16) && out_stride * ob % 16 == 0 && n * ob % 16 == 0;
  CUtensorMap a_map, a_part_map;
  if (!make_map(&a_map, a, 1, rows, k, a_stride, kTileM) ||
      !make_map(&a_part_map, a, 1, rows, k, a_stride, kRowBox))
    return refused();
  CUtensorMap out_map = a_map;  // not used unless P.tma_out
  if (P.tma_out && !make_map(&out_map, out, ob, rows, n, out_stride * ob, 32)) return refused();
  const auto launch = [&](auto t, auto tile_n, auto share, int cluster) -> tbe_status {
    using T = decltype(t);
    constexpr int kTileN = decltype(tile_n)::value;
    constexpr Share kShare = decltype(share)::value;
    using Shape = ProductShape<kTileN, kShare>;
    P.n_tiles = static_cast<int>((n + kTileN - 1) / kTileN);
    CUtensorMap w_map;
    if (!make_map(&w_map, w, 1, static_cast<int64_t>(experts) * n, k, k, Shape::kWRows))
      return refused();
    const auto kernel = product_kernel<T, kTileN, kShare>;
    constexpr int kSmem = Shape::kSmem;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
        cudaSuccess)
      return refused();
    P.row_tiles = static_cast<int>(most_row_tiles(rows, experts, Shape::kTileRows));
    const int64_t most = static_cast<int64_t>(P.row_tiles) * P.n_tiles;
    if (most > INT32_MAX / 8) return TBE_EUNSUPPORTED;  // the kernel counts tiles in 32 bits
    const int64_t room = sms / cluster;
    const int64_t clusters = kShare == kSplit || most < room ? most : room;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster));
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    // its start may overlap the end of the kernel before it (griddepcontrol.wait)
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a_map, a_part_map, w_map, out_map, P) != cudaSuccess)
      return refused();
    return launched();
  };
  using Narrow = std::integral_constant<int, 128>;
  using Wide = std::integral_constant<int, 256>;
  using Alone = std::integral_constant<Share, kAlone>;
  using Pair = std::integral_constant<Share, kPair>;
  using Split = std::integral_constant<Share, kSplit>;
  return for_dtype(out_dtype, [&](auto t) {
    const ProductForm form = product_form(rows, n, P.kb, experts, sms);
    if (form.share == kSplit) return launch(t, Narrow{}, Split{}, form.cluster);
    if (form.share == kAlone) return launch(t, Narrow{}, Alone{}, form.cluster);
    return launch(t, Wide{}, Pair{}, form.cluster);
  });
}
