// Token embedding: a row of a table for each token, and the table's gradient by
// sorted tokens.  The operations are specified in include/tbe_embed.h.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "entry.cuh"
#include "sort.cuh"
#include "tbe_embed.h"

namespace tbe {
namespace {

// -------------------------------------------------------------------- lookup
//
// Memory bounds it (131072 tokens of 131072 rows, 2048 bf16: 110 us, 6.1 TB/s of what must move).
// A group of `1 << log_group` threads carries a token's row, up to four 16-byte vectors in
// flight a thread; rows off 16-byte boundaries go in vectors all the same (inner_span,
// load_vec).
constexpr int kMoveThreads = 256;
constexpr int kInFlight = 4;

template <typename T, typename IdT, bool kAligned>
__global__ void __launch_bounds__(kMoveThreads)
    embed_kernel(const T* __restrict__ table, int rows, int width, int64_t table_stride,
                 const IdT* __restrict__ ids, int tokens, float scale, T* __restrict__ out,
                 int64_t out_stride, int log_group) {
  constexpr int V = kVec<T>;
  const int size = 1 << log_group, t = threadIdx.x & (size - 1);
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (kMoveThreads >> log_group) +
                        (threadIdx.x >> log_group);
  if (token >= tokens) return;
  const IdT id = ids[token];
  const bool on = id >= 0 && id < static_cast<IdT>(rows);
  const T* src = table + (on ? static_cast<int64_t>(id) * table_stride : 0);
  T* dst = out + token * out_stride;
  const Span s = inner_span<T, kAligned>(dst, width);
  for (int e0 = s.lo + t * V; e0 < s.hi; e0 += size * V * kInFlight) {
    Pack<T, V> v[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (on && e0 + u * size * V < s.hi) v[u] = load_vec<T, kAligned>(src + e0 + u * size * V);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      if (e0 + u * size * V >= s.hi) continue;
      float f[V] = {};
      if (on) {
        to_floats<T>(v[u], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= scale;
      }
      store_vec(dst + e0 + u * size * V, from_floats<T>(f));
    }
  }
  if constexpr (!kAligned)
    for_ends(s, width, t, size,
             [&](int e) { dst[e] = from_f32<T>(on ? scale * to_f32(src[e]) : 0.f); });
}

// ---------------------------------------------------------------------- sort
//
// Tokens sorted by row, stably, as items (row, token); tokens without a row get row V, which
// comes last.  A radix sort from the lowest digit, each pass a counting sort
// as the experts' (a warp counts its run of the items in its own row of shared memory, the
// rows are scanned, and the warp walks its run again).  Up to kOneLaunch tokens (kOneCleared where
// the result is cleared beside it) all passes are one launch of one cluster; above, three
// launches a pass over the whole GPU.  Both measured, with 100000 rows (two passes), gradients of
// 256 columns added: 65536 tokens 39 us in one launch and 45 in six, 98304 52 and 51, 131072 66 and
// 59; of 1024 columns stored: 98304 tokens 97 and 113, 131072 117 and 127, 196608 154 and 151.
constexpr int kDigitBits = 10;  // of a pass, at most
constexpr int kSortUnroll = 4;
constexpr int kOneLaunch = 98304, kOneCleared = 163840;
constexpr int kTokensPerCta = 1024;   // another CTA's share (4097 tokens: 10.9 us, with 2048 12.8)
constexpr int kGridCtas = 304;
constexpr int kGridChunk = 4096;      // items of a CTA of three launches, at least

struct Item {
  int row, token;
};

template <typename IdT>
struct FromIds {
  const IdT* ids;
  int rows;
  __device__ __forceinline__ Item operator()(int64_t i) const {
    const IdT id = ids[i];
    return {id >= 0 && id < static_cast<IdT>(rows) ? static_cast<int>(id) : rows,
            static_cast<int>(i)};
  }
};
// Past the first pass: items that other multiprocessors wrote in this launch (read from L2).
struct FromItems {
  const Item* items;
  __device__ __forceinline__ Item operator()(int64_t i) const {
    const int2 v = __ldcg(reinterpret_cast<const int2*>(items + i));
    return {v.x, v.y};
  }
};

struct Digit {
  int shift, bits;
  __device__ __forceinline__ int buckets() const { return 1 << bits; }
  __device__ __forceinline__ int of(const Item& it) const {
    return (it.row >> shift) & (buckets() - 1);
  }
};

// Every warp's counts of its run, count[warp][bucket], and total[bucket].  The whole
// CTA; ends before a barrier.
template <typename Source>
__device__ __forceinline__ void count_items(const Source& from, Chunk c, Digit d, int* count,
                                            int* total) {
  const int buckets = d.buckets(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * buckets; i += blockDim.x) count[i] = 0;
  __syncthreads();
  int* mine = count + warp * buckets;
  for (int64_t a0 = c.first + lane; a0 < c.last; a0 += 32 * kSortUnroll) {
    Item it[kSortUnroll];
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u)
      if (a0 + 32 * u < c.last) it[u] = from(a0 + 32 * u);
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u)
      if (a0 + 32 * u < c.last) atomicAdd(mine + d.of(it[u]), 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < buckets; e += blockDim.x) {
    int sum = 0;
#pragma unroll 16
    for (int w = 0; w < kSortWarps; ++w) sum += count[w * buckets + e];
    total[e] = sum;
  }
}

template <typename Source>
__device__ __forceinline__ void place_items(const Source& from, Chunk c, Digit d, int* mine,
                                            Item* to) {
  const int lane = threadIdx.x & 31;
  for (int64_t a0 = c.first; a0 < c.last; a0 += 32 * kSortUnroll) {
    Item it[kSortUnroll];
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u)
      if (a0 + 32 * u + lane < c.last) it[u] = from(a0 + 32 * u + lane);
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      const bool on = a0 + 32 * u + lane < c.last;
      const int b = on ? d.of(it[u]) : -1;
      const unsigned same = __match_any_sync(kAll, b);
      int place = 0;
      if (on) place = mine[b] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (on && (same >> lane) == 1u) mine[b] = place + 1;  // the highest lane of its bucket
      __syncwarp();
      if (on) to[place] = it[u];
    }
  }
}

// One pass in a cluster: smem holds total[buckets], then count[kSortWarps][buckets].
template <typename Source>
__device__ __forceinline__ void cluster_pass(const Source& from, int n, Digit d, int* smem,
                                             int* warp_sum, Item* to) {
  const int buckets = d.buckets(), ctas = gridDim.x, rank = blockIdx.x;
  int *total = smem, *count = smem + buckets;
  const int64_t per_warp = (static_cast<int64_t>(n) + ctas * kSortWarps * 32 - 1) /
                           (ctas * kSortWarps * 32) * 32;
  const Chunk chunk = warp_chunk(n, rank * kSortWarps * per_warp, per_warp);
  count_items(from, chunk, d, count, total);
  cluster_arrive();
  cluster_wait();
  // a bucket a thread: no digit has more buckets than the CTA threads
  const int e = threadIdx.x;
  int all = 0, before = 0;
  if (e < buckets) {
    int c[kSortMostCtas];
#pragma unroll
    for (int r = 0; r < kSortMostCtas; ++r) c[r] = r < ctas ? load_from_cta(total + e, r) : 0;
#pragma unroll
    for (int r = 0; r < kSortMostCtas; ++r) {
      all += c[r];
      before += r < rank ? c[r] : 0;
    }
  }
  int sum;
  const int at = block_scan(all, warp_sum, &sum);
  if (e < buckets) counts_to_places(count, buckets, e, at + before);
  __syncthreads();
  place_items(from, chunk, d, count + (threadIdx.x >> 5) * buckets, to);
  // the items are there for the other CTAs, and no totals are read any more
  cluster_arrive();
  cluster_wait();
}

struct SortPlan {
  int n, rows, passes, bits;  // bits of a digit
  Item* items[2];             // pass p writes items[p % 2]
};

template <typename IdT>
__global__ void __launch_bounds__(kSortWarps * 32)
    token_sort_kernel(const IdT* __restrict__ ids, const SortPlan plan) {
  extern __shared__ int sort_smem[];
  __shared__ int warp_sum[kSortWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cluster_pass(FromIds<IdT>{ids, plan.rows}, plan.n, Digit{0, plan.bits}, sort_smem, warp_sum,
               plan.items[0]);
  for (int p = 1; p < plan.passes; ++p)
    cluster_pass(FromItems{plan.items[(p + 1) & 1]}, plan.n, Digit{p * plan.bits, plan.bits},
                 sort_smem, warp_sum, plan.items[p & 1]);
}

// The three launches of a pass: totals[cta][bucket], turned into the bucket's items in the
// CTAs before, and sums[bucket].
template <typename Source>
__global__ void __launch_bounds__(kSortWarps * 32)
    token_count_kernel(const Source from, int n, Digit d, int* __restrict__ totals) {
  extern __shared__ int sort_smem[];
  const int buckets = d.buckets();
  count_items(from, my_chunk(n), d, sort_smem + buckets, sort_smem);
  for (int e = threadIdx.x; e < buckets; e += blockDim.x)  // the entries it summed: no barrier
    totals[static_cast<int64_t>(blockIdx.x) * buckets + e] = sort_smem[e];
}

// A warp a bucket, lane l over a run of the CTAs.
__global__ void __launch_bounds__(256)
    token_scan_kernel(int* __restrict__ totals, int ctas, int buckets, int* __restrict__ sums) {
  constexpr int kMost = (kGridCtas + 31) / 32;
  const int b = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= buckets) return;
  const int per = (ctas + 31) / 32;
  int v[kMost], sum = 0;
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    const int c = lane * per + j;
    v[j] = j < per && c < ctas ? totals[static_cast<int64_t>(c) * buckets + b] : 0;
    sum += v[j];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += y;
  }
  int at = incl - sum;
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    const int c = lane * per + j;
    if (j < per && c < ctas) totals[static_cast<int64_t>(c) * buckets + b] = at;
    at += v[j];
  }
  if (lane == 31) sums[b] = incl;
}

template <typename Source>
__global__ void __launch_bounds__(kSortWarps * 32)
    token_place_kernel(const Source from, int n, Digit d, const int* __restrict__ totals,
                       const int* __restrict__ sums, Item* __restrict__ to) {
  extern __shared__ int sort_smem[];
  __shared__ int warp_sum[kSortWarps];
  const int buckets = d.buckets(), e = threadIdx.x;
  int* count = sort_smem + buckets;
  const Chunk chunk = my_chunk(n);
  count_items(from, chunk, d, count, sort_smem);
  int sum;
  const int at = block_scan(e < buckets ? sums[e] : 0, warp_sum, &sum);
  if (e < buckets)
    counts_to_places(count, buckets, e,
                     at + totals[static_cast<int64_t>(blockIdx.x) * buckets + e]);
  __syncthreads();
  place_items(from, chunk, d, count + (threadIdx.x >> 5) * buckets, to);
}

// ------------------------------------------------------------------ gradient
//
// The sorted items are cut into pieces of `piece` places.  A group of threads sums the runs
// of equal rows that begin in its piece, a vector of columns a thread, and writes their
// rows.  A run that crosses a boundary belongs to the piece it begins in, which follows it into
// the next one; but where it crosses two boundaries it is long, and each of its pieces leaves
// its part: slot 0 where the run began before the piece, slot 1 where it begins in it.  A second
// launch adds those parts in the pieces' order.  Rows without tokens are cleared before.
//
// What bounds it is how many rows' loads are on their way, so each thread copies its own columns of
// the next rows to a ring in shared memory (cp.async) while it adds the row at hand (65536 tokens,
// 2048 bf16: 62 us, 6.1 TB/s; with eight rows at a time in registers 98).
constexpr int kLeastPiece = 8, kMostPiece = 64;
constexpr int64_t kSumThreads = 152 * 2048;  // threads that fill the GPU
constexpr int kJoinPieces = 32;       // pieces whose ends a CTA looks at, at most
constexpr int kJoinSegments = 8;
constexpr int kJoinLanes = 32;        // vectors of four columns of a CTA

struct SumArgs {
  const void* grad_out;
  const Item* items;
  void* out;
  float* parts;  // [pieces][2][part_width]
  int64_t grad_stride, out_stride;
  int n, rows, width, part_width, piece, join;  // join: pieces of a joining CTA
  float scale;
  bool accumulate;
};

__device__ __forceinline__ Item item_at(const Item* items, int64_t i) {
  const int2 v = *reinterpret_cast<const int2*>(items + i);
  return {v.x, v.y};
}

// Rounds N sums into columns col .. of a row of the result.
template <typename O, int N, bool kAligned>
__device__ __forceinline__ void store_sums(const SumArgs& P, int row, int col,
                                           const float (&sum)[N]) {
  O* to = static_cast<O*>(P.out) + static_cast<int64_t>(row) * P.out_stride + col;
  if constexpr (kAligned) {
#pragma unroll
    for (int c = 0; c < N; c += kVec<O>) {
      float f[kVec<O>] = {};
      if (P.accumulate) to_floats<O>(*reinterpret_cast<const Pack<O, kVec<O>>*>(to + c), f);
#pragma unroll
      for (int i = 0; i < kVec<O>; ++i) f[i] = fmaf(P.scale, sum[c + i], f[i]);
      store_vec(to + c, from_floats<O>(f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (col + i < P.width)
        to[i] = from_f32<O>(fmaf(P.scale, sum[i], P.accumulate ? to_f32(to[i]) : 0.f));
  }
}

// Whether the run of `row` that crosses the boundary `at` between two pieces crosses the boundary
// before or behind it too.  row_at(i): the row of the i-th place.
template <typename RowAt>
__device__ __forceinline__ bool is_long(const SumArgs& P, int64_t at, int row, RowAt row_at) {
  return (at + P.piece < P.n && row_at(at + P.piece) == row) ||
         (at > P.piece && row_at(at - P.piece - 1) == row);
}

// Rows of grad_out on their way to a thread: its vector of each, or where rows are off 16
// bytes, the two aligned vectors around it.  (16 bytes that hold a byte of a row lie in its
// allocation; what is not the row's is not used.)
template <typename T, bool kAligned>
struct RowsAhead {
  static constexpr int V = kVec<T>, kSlots = kAligned ? 1 : 2;
  static constexpr int kDeep = kAligned ? 8 : 6;
  static constexpr int kBytes = kDeep * kSlots * 16;  // a thread
  uint4* slots;  // this thread's first; the CTA's threads lie side by side

  __device__ __forceinline__ uint4* slot(int stage, int k) const {
    return slots + (stage * kSlots + k) * kMoveThreads;
  }
  // at: the thread's first column of a row, `left` columns before its end.
  __device__ __forceinline__ void start(int stage, const T* at, int left) const {
    if constexpr (kAligned) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<unsigned>(
                       __cvta_generic_to_shared(slot(stage, 0)))),
                   "l"(at)
                   : "memory");
    } else {
      const int before = lead<T>(at);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (k * V - before < left)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(static_cast<unsigned>(
                           __cvta_generic_to_shared(slot(stage, k)))),
                       "l"(at - before + k * V)
                       : "memory");
    }
  }
  static __device__ __forceinline__ void close() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // All but the last kDeep - 1 rows are there.
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
  }
  // The thread's columns, which begin `bytes` past a boundary; what lies past the row's end is not
  // defined.
  __device__ __forceinline__ Pack<T, V> read(int stage, int bytes) const {
    if constexpr (kAligned) {
      return *reinterpret_cast<const Pack<T, V>*>(slot(stage, 0));
    } else {
      const uint4 o = cut_row(*slot(stage, 0), *slot(stage, 1), bytes);
      return *reinterpret_cast<const Pack<T, V>*>(&o);
    }
  }
};

extern __shared__ uint4 embed_ring[];

template <typename T, typename O, bool kAligned>
__global__ void __launch_bounds__(kMoveThreads)
    embed_sum_kernel(const __grid_constant__ SumArgs P, int log_group) {
  constexpr int V = kVec<T>;
  using Ring = RowsAhead<T, kAligned>;
  const int groups = kMoveThreads >> log_group;
  const int size = 1 << log_group, t = threadIdx.x & (size - 1);
  // the items of the CTA's pieces, of the one before and of the one behind
  Item* window = reinterpret_cast<Item*>(embed_ring + Ring::kDeep * Ring::kSlots * kMoveThreads);
  const int64_t piece0 = static_cast<int64_t>(blockIdx.x) * groups;
  const int64_t base = (piece0 - 1) * P.piece - 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < (groups + 2) * P.piece + 2; i += kMoveThreads)
    window[i] = base + i >= 0 && base + i < P.n ? item_at(P.items, base + i) : Item{P.rows, 0};
  __syncthreads();
  const auto row_at = [&](int64_t i) { return window[i - base].row; };

  const int64_t piece = piece0 + (threadIdx.x >> log_group);
  const int col = (blockIdx.y * size + t) * V;
  const int64_t first = piece * P.piece;
  if (first >= P.n || col >= P.width) return;
  const int64_t last = first + P.piece < P.n ? first + P.piece : P.n;
  const Item *at = window + (first - base), *end = window + (last - base);
  if (at->row >= P.rows) return;
  bool open = false;  // the first run has a part before this one
  if (first > 0 && row_at(first - 1) == at->row) {
    open = is_long(P, first, at->row, row_at);
    if (!open)  // the piece before sums it
      for (const int skip = at->row; at < end && at->row == skip;) ++at;
  }
  const int tail = end[-1].row;
  bool leaves = false;  // the last run's part goes on in the next piece
  if (last < P.n && tail < P.rows && end->row == tail) {
    leaves = is_long(P, last, tail, row_at);
    if (!leaves)  // at most a piece on
      for (const Item* n = window + (P.n - base); end < n && end->row == tail;) ++end;
  }
  while (at < end && end[-1].row >= P.rows) --end;  // tokens without a row come last
  if (at == end) return;

  const T* grad = static_cast<const T*>(P.grad_out) + col;
  const Ring ring = {embed_ring + threadIdx.x};
  const auto start = [&](int stage, const Item* i) {
    if (i < end) ring.start(stage, grad + i->token * P.grad_stride, P.width - col);
    ring.close();
  };
#pragma unroll
  for (int k = 0; k < Ring::kDeep; ++k) start(k, at + k);

  float2 sum[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) sum[i] = make_float2(0.f, 0.f);
  const auto leave = [&](int slot) {
    float* parts = P.parts + (piece * 2 + slot) * P.part_width + col;
#pragma unroll
    for (int i = 0; i < V / 2; i += 2)
      *reinterpret_cast<float4*>(parts + 2 * i) =
          make_float4(sum[i].x, sum[i].y, sum[i + 1].x, sum[i + 1].y);
  };
  const auto finish = [&](int row) {  // the run ends here
    if (open) {
      leave(0);
    } else {
      float f[V];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) f[2 * i] = sum[i].x, f[2 * i + 1] = sum[i].y;
      store_sums<O, V, kAligned>(P, row, col, f);
    }
    open = false;
  };
  int run = at->row, stage = 0;
  for (;;) {
    const Item it = *at;
    if (it.row != run) {
      finish(run);
      run = it.row;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) sum[i] = make_float2(0.f, 0.f);
    }
    ring.wait();
    float f[V];
    // a row's distance from a boundary, in arithmetic modulo 2^32
    const int bytes = static_cast<int>(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(grad)) +
                                       static_cast<uint32_t>(it.token) *
                                           static_cast<uint32_t>(P.grad_stride * sizeof(T))) & 15;
    to_floats<T>(ring.read(stage, bytes), f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      sum[i] = __fadd2_rn(sum[i], make_float2(f[2 * i], f[2 * i + 1]));
    start(stage, at + Ring::kDeep);
    stage = stage + 1 == Ring::kDeep ? 0 : stage + 1;
    if (++at == end) break;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (leaves) leave(open ? 0 : 1);
  else finish(run);
}

// Adds the parts of the long runs.  A CTA looks at the ends of P.join pieces, a lane each,
// for long runs that begin before them, and forms kJoinLanes * 4 columns of each, the
// run's pieces shared by kJoinSegments segments of threads.
template <typename O>
__global__ void __launch_bounds__(kJoinLanes * kJoinSegments)
    embed_join_kernel(const __grid_constant__ SumArgs P) {
  __shared__ float4 sums[kJoinSegments][kJoinLanes];
  const int lane = threadIdx.x & 31, segment = threadIdx.x / kJoinLanes;
  const int col = (blockIdx.y * kJoinLanes + threadIdx.x % kJoinLanes) * 4;
  const bool on = col < P.part_width;
  const auto row_at = [&](int64_t i) { return i < P.n ? item_at(P.items, i).row : P.rows; };
  const int64_t piece0 = static_cast<int64_t>(blockIdx.x) * P.join;
  const int64_t end = (piece0 + lane + 1) * P.piece;
  const int run_here = lane < P.join ? row_at(end) : P.rows;
  const bool found = run_here < P.rows && row_at(end - 1) == run_here &&
                     (end == P.piece || row_at(end - P.piece - 1) != run_here) &&
                     is_long(P, end, run_here, row_at);
  bool waited = false;
  for (unsigned todo = __ballot_sync(kAll, found); todo; todo &= todo - 1) {
    const int64_t piece = piece0 + __ffs(todo) - 1;
    const int run = __shfl_sync(kAll, run_here, __ffs(todo) - 1);
    int more = 0;  // pieces behind, looked through 32 at a time
    for (unsigned all = kAll; all == kAll;) {
      all = __ballot_sync(kAll, row_at((piece + 1 + more + lane) * P.piece) == run);
      more += __popc(all);
    }
    // The items were there when the sums began; the sums' parts and rows are from here on.
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    waited = true;
    const auto part = [&](int64_t p, int slot) {
      return *reinterpret_cast<const float4*>(P.parts + (p * 2 + slot) * P.part_width + col);
    };
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](float4 v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    if (on) {
#pragma unroll 8
      for (int k = 1 + segment; k <= more; k += kJoinSegments) add(part(piece + k, 0));
    }
    __syncthreads();  // the sums of the run before have been read
    sums[segment][threadIdx.x % kJoinLanes] = s;
    __syncthreads();
    if (segment == 0 && on) {
      s = part(piece, 1);
#pragma unroll
      for (int i = 0; i < kJoinSegments; ++i) add(sums[i][threadIdx.x]);
      const float v[4] = {s.x, s.y, s.z, s.w};
      store_sums<O, 4, false>(P, run, col, v);
    }
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the call ends after its sums
}

// -------------------------------------------------------- gradient, few tokens
//
// In one launch, without a sort: every CTA reads all ids.  The first CTAs have a token each, and
// the one with a row's first token lists the row's tokens in their order and sums them; a
// CTA's groups of threads take equal parts of a long list, added in their order.  The other
// CTAs clear the rows of their range that have no token.  64 tokens of 1000 rows x 1024 bf16 take
// 3.8 us and sorted 13; 1024 of 5000 rows 9.4 and about 18, 2048 18 both.  A list as long as the
// tokens is slower (1024 tokens of one row: 39 us, sorted 19), which sets the limit, and with
// 128 threads a row rather than 256 there are more CTAs for its columns (x 2048: 41 us and 74;
// 1024 tokens of 5000 rows 15 and 11).
constexpr int kFewTokens = 1024;
constexpr int kFewLog = 7;        // log of the threads of a row, at most
constexpr int kFewRows = 32768;  // of a clearing CTA, at most: a bit each in its shared memory

template <typename IdT>
struct FewArgs {
  SumArgs sum;  // of which items, parts, part_width and piece are not used
  const IdT* ids;
  int range;  // rows of a clearing CTA
};

template <typename T, typename O, typename IdT, bool kAligned>
__global__ void __launch_bounds__(kMoveThreads)
    embed_few_kernel(const __grid_constant__ FewArgs<IdT> A, int log_group) {
  constexpr int V = kVec<T>, kInBatch = 16;
  const SumArgs& P = A.sum;
  __shared__ int list[kFewTokens];
  __shared__ unsigned found[kFewTokens / 32];
  extern __shared__ float few_sums[];  // [groups][size * V]
  const FromIds<IdT> from = {A.ids, P.rows};
  const int groups = kMoveThreads >> log_group, size = 1 << log_group;
  const int group = threadIdx.x >> log_group, t = threadIdx.x & (size - 1);
  const int lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) >= P.n) {
    const int64_t r0 = (static_cast<int64_t>(blockIdx.x - P.n) * gridDim.y + blockIdx.y) * A.range;
    if (r0 >= P.rows) return;
    const int rows = static_cast<int>(P.rows - r0 < A.range ? P.rows - r0 : A.range);
    // which of them have tokens, a bit each
    unsigned* has = reinterpret_cast<unsigned*>(few_sums);
    for (int i = threadIdx.x; i < (A.range + 31) / 32; i += kMoveThreads) has[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < P.n; i += kMoveThreads) {
      const int64_t r = from(i).row - r0;
      if (r >= 0 && r < rows) atomicOr(has + (r >> 5), 1u << (r & 31));
    }
    __syncthreads();
    Pack<O, kVec<O>> zero;
#pragma unroll
    for (int i = 0; i < kVec<O>; ++i) zero.v[i] = from_f32<O>(0.f);
    for (int r = group; r < rows; r += groups) {
      if (has[r >> 5] >> (r & 31) & 1) continue;
      O* row = static_cast<O*>(P.out) + (r0 + r) * P.out_stride;
      const Span s = inner_span<O, kAligned>(row, P.width);
      for (int e = s.lo + t * kVec<O>; e < s.hi; e += size * kVec<O>) store_vec(row + e, zero);
      for_ends(s, P.width, t, size, [&](int e) { row[e] = from_f32<O>(0.f); });
    }
    return;
  }
  const int token = blockIdx.x, run = from(token).row;
  if (run >= P.rows) return;
  bool before = false;
  for (int i0 = 0; i0 < P.n; i0 += kMoveThreads) {
    const int i = i0 + threadIdx.x;
    const bool same = i < P.n && from(i).row == run;
    before |= same && i < token;
    const unsigned all = __ballot_sync(kAll, same);
    if (lane == 0 && i < kFewTokens) found[i >> 5] = all;
  }
  if (__syncthreads_or(before)) return;  // an earlier token's CTA does it
  int count = 0;
  for (int w = 0; w < (P.n + 31) / 32; ++w) {
    const unsigned all = found[w];
    if (w % (kMoveThreads / 32) == static_cast<int>(threadIdx.x >> 5) && all >> lane & 1)
      list[count + __popc(all & ((1u << lane) - 1))] = w * 32 + lane;
    count += __popc(all);
  }
  __syncthreads();
  // this group's part of the list
  const int per = (count + groups - 1) / groups, first = group * per;
  const int last = first + per < count ? first + per : count;
  const int col = (blockIdx.y * size + t) * V;
  const T* grad = static_cast<const T*>(P.grad_out);
  float sum[V] = {};
  for (int i0 = first; i0 < last && col < P.width; i0 += kInBatch) {
    Pack<T, V> v[kInBatch];
#pragma unroll
    for (int u = 0; u < kInBatch; ++u) {
      if (i0 + u >= last) break;
      const T* row = grad + list[i0 + u] * P.grad_stride;
      if constexpr (kAligned) {
        v[u] = load_vec<T, true>(row + col);
      } else if (col >= V && col + 2 * V <= P.width) {
        v[u] = load_vec<T, false>(row + col);  // the aligned vectors around it lie in the row
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[u].v[i] = col + i < P.width ? row[col + i] : from_f32<T>(0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < kInBatch; ++u) {
      if (i0 + u >= last) break;
      float f[V];
      to_floats<T>(v[u], f);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += f[i];
    }
  }
  if (count > 1 && groups > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) few_sums[(group * V + i) * size + t] = sum[i];
    __syncthreads();
    if (group == 0)
      for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += few_sums[(g * V + i) * size + t];
  }
  if (group == 0 && col < P.width) store_sums<O, V, kAligned>(P, run, col, sum);
}

// Zeros: rows of `bytes` bytes, `pitch` apart, the last of `last` bytes; `unit` bytes divide
// them all.  May run beside the sort, whose end it waits for before its own.
__global__ void __launch_bounds__(kMoveThreads)
    clear_kernel(char* p, int64_t rows, int64_t bytes, int64_t pitch, int64_t last, int unit) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    char* row = p + r * pitch;
    char* end = row + (r + 1 < rows ? bytes : last);
    char* lo = row + (-reinterpret_cast<uintptr_t>(row) & 15);
    if (lo > end) lo = end;
    char* hi = lo + ((end - lo) & ~int64_t(15));
    for (char* q = lo + threadIdx.x * 16; q < hi; q += kMoveThreads * 16)
      *reinterpret_cast<uint4*>(q) = make_uint4(0, 0, 0, 0);
    const int64_t ends = (lo - row) + (end - hi);  // less than 32 bytes
    if (static_cast<int64_t>(threadIdx.x) * unit < ends) {
      const int64_t at = threadIdx.x * unit;
      char* q = at < lo - row ? row + at : hi + (at - (lo - row));
      if (unit == 2) *reinterpret_cast<uint16_t*>(q) = 0;
      else *reinterpret_cast<uint32_t*>(q) = 0;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// -------------------------------------------------------------- host

constexpr int64_t kMost = INT32_MAX - 1024;  // tokens and rows, counted in 32 bits
constexpr int64_t kMostWidth = int64_t(1) << 20;

int log2_up(int64_t n) {
  int lg = 0;
  while ((int64_t(1) << lg) < n) ++lg;
  return lg;
}

SortPlan plan_of(int64_t tokens, int64_t rows) {
  SortPlan p = {};
  p.n = static_cast<int>(tokens);
  p.rows = static_cast<int>(rows);
  const int bits = std::max(1, log2_up(rows + 1));  // of the rows and the one past them
  p.passes = (bits + kDigitBits - 1) / kDigitBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  return p;
}

// Places of a piece: few while that leaves the GPU idle (4097 tokens, 1001 fp16: sums 9.4 us in
// pieces of 8, 21 in pieces of 32), more as the tokens are more, since a long run has a part in
// each.
int64_t piece_of(int64_t tokens, int64_t width) {
  const int64_t threads = std::min<int64_t>((width + 7) / 8, 256);  // of a piece, about
  int64_t piece = kLeastPiece;
  while (piece < kMostPiece && tokens * threads >= 2 * piece * kSumThreads) piece *= 2;
  return piece;
}

// The workspace's parts, in bytes from its start.
struct Layout {
  int64_t items[2], totals, sums, parts, bytes;
};
Layout layout_of(int64_t tokens, int64_t width) {
  const auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  Layout l = {};
  if (tokens <= kFewTokens) return l;
  l.items[1] = up(tokens * 8);
  l.totals = l.items[1] + up(tokens * 8);
  l.sums = l.totals + (tokens > kOneLaunch ? up(int64_t(kGridCtas) * 4 << kDigitBits) : 0);
  l.parts = l.sums + (tokens > kOneLaunch ? up(int64_t(4) << kDigitBits) : 0);
  const int64_t piece = piece_of(tokens, width), pieces = (tokens + piece - 1) / piece;
  l.bytes = l.parts + pieces * 2 * ((width + 7) / 8 * 8) * 4;
  return l;
}

tbe_status check_sizes(int64_t tokens, int64_t rows, int64_t width) {
  if (tokens < 0 || rows < 0 || width < 0) return TBE_EINVAL;
  return tokens >= kMost || rows >= kMost || width > kMostWidth ? TBE_EUNSUPPORTED : TBE_OK;
}

bool check_ids(const void* ids, int32_t dtype, int64_t tokens) {
  return !tokens || (ids && aligned_to(ids, dtype == TBE_DT_I32 ? 4 : 8));
}

// Room for a kernel's launches in shared memory; most: of the largest of them.  It belongs to the
// kernel, so a launch that asked for its own size could take from another, which a second host
// thread may be about to make or a graph holds.
cudaError_t room_for(const void* kernel, size_t most) {
  return most <= 40 * 1024 ? cudaSuccess  // beside what is declared in the kernels
                           : cudaFuncSetAttribute(kernel,
                                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  static_cast<int>(most));
}

template <typename IdT>
tbe_status sort_in_cluster(const IdT* ids, const SortPlan& plan, cudaStream_t s) {
  const auto kernel = token_sort_kernel<IdT>;
  int ctas = 1;
  while (ctas < kSortMostCtas && plan.n > ctas * kTokensPerCta) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kSortWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(kSortWarps + 1) * 4 << plan.bits;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (room_for(reinterpret_cast<const void*>(kernel),
               static_cast<size_t>(kSortWarps + 1) * 4 << kDigitBits) != cudaSuccess ||
      (ctas > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                        1) != cudaSuccess) ||
      cudaLaunchKernelEx(&cfg, kernel, ids, plan) != cudaSuccess)
    return refused();
  return launched();
}

template <typename Source>
tbe_status sort_pass(const Source& from, const SortPlan& plan, int p, int* totals, int* sums,
                     cudaStream_t s) {
  const Digit d = {p * plan.bits, plan.bits};
  const int buckets = 1 << plan.bits, ctas = std::min(plan.n / kGridChunk, kGridCtas);
  const size_t smem = static_cast<size_t>(kSortWarps + 1) * 4 << plan.bits;
  const size_t most = static_cast<size_t>(kSortWarps + 1) * 4 << kDigitBits;
  if (room_for(reinterpret_cast<const void*>(token_count_kernel<Source>), most) != cudaSuccess ||
      room_for(reinterpret_cast<const void*>(token_place_kernel<Source>), most) != cudaSuccess)
    return refused();
  token_count_kernel<Source><<<ctas, kSortWarps * 32, smem, s>>>(from, plan.n, d, totals);
  note_launch();
  token_scan_kernel<<<(buckets + 7) / 8, 256, 0, s>>>(totals, ctas, buckets, sums);
  note_launch();
  token_place_kernel<Source>
      <<<ctas, kSortWarps * 32, smem, s>>>(from, plan.n, d, totals, sums, plan.items[p & 1]);
  return launched();
}

template <typename IdT>
tbe_status sort_in_grid(const IdT* ids, const SortPlan& plan, int* totals, int* sums,
                        cudaStream_t s) {
  tbe_status st = sort_pass(FromIds<IdT>{ids, plan.rows}, plan, 0, totals, sums, s);
  for (int p = 1; st == TBE_OK && p < plan.passes; ++p)
    st = sort_pass(FromItems{plan.items[(p + 1) & 1]}, plan, p, totals, sums, s);
  return st;
}

// A launch with `smem` bytes of the `most` that the kernel is ever launched with; with `beside` it
// may begin before the kernel ahead of it ends, and waits for that one's results itself.
template <typename... Args>
tbe_status launch(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, size_t most,
                  bool beside, cudaStream_t s, std::common_type_t<Args>... args) {
  if (room_for(reinterpret_cast<const void*>(kernel), most) != cudaSuccess) return refused();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return refused();
  note_launch();
  return TBE_OK;
}

// Zeros in a matrix.  Beside the cluster that sorts, six CTAs a multiprocessor are all resident;
// more would wait for the cluster's end, with a CTA's whole share still to do (eight: 131 MB and
// 8192 tokens 39.6 us instead of 34.0, 537 MB and 65536 tokens 177 instead of 154), or at sixteen
// with less of it, which pays for large results (537 MB 150 us, 1.07 GB 303 and 319 with six; 268 MB
// 68 and 66).
tbe_status clear(void* p, int64_t rows, int64_t width, int64_t stride, int bytes, bool beside,
                 cudaStream_t s) {
  int64_t row = width * bytes, pitch = stride * bytes, last = row;
  if (pitch == row) {  // one block of memory: rows of 32 KB
    const int64_t all = rows * row;
    pitch = row = 32768;
    rows = (all + row - 1) / row;
    last = all - (rows - 1) * row;
  }
  const int per_sm = beside && rows * row < (400 << 20) ? 6 : 16;
  return launch(clear_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(rows, 152 * per_sm))),
                kMoveThreads, 0, 0, beside, s, static_cast<char*>(p), rows, row, pitch, last,
                bytes);
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_embed(const void* table, int32_t dtype, int64_t rows, int64_t width,
                                int64_t table_stride, const void* ids, int32_t index_dtype,
                                int64_t tokens, float scale, void* out, int64_t out_stride,
                                void* stream) {
  const tbe_status bad = check_sizes(tokens, rows, width);
  if (bad != TBE_OK) return bad;
  if (!dtype_bytes(dtype) || (index_dtype != TBE_DT_I32 && index_dtype != TBE_DT_I64))
    return TBE_EUNSUPPORTED;
  if (!std::isfinite(scale)) return TBE_EINVAL;
  if (!tokens || !width) return TBE_OK;
  const int b = dtype_bytes(dtype);
  const Matrix in = {table, table_stride, b}, to = {out, out_stride, b};
  if ((rows && !in.good(rows, width)) || !to.good(tokens, width) ||
      !check_ids(ids, index_dtype, tokens) ||
      overlap(in.span(rows, width), to.span(tokens, width)) ||
      overlap(run_of(ids, tokens * (index_dtype == TBE_DT_I32 ? 4 : 8)), to.span(tokens, width)))
    return TBE_EINVAL;
  const bool vec = (!rows || in.vectors(width, 16)) && to.vectors(width, 16);
  return for_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const auto go = [&](auto aligned, auto* p) {
      constexpr bool kAligned = decltype(aligned)::value;
      using IdT = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
      // A thread for each vector while the tokens are few and latency counts, one for four
      // once they fill the GPU.
      int64_t places = (width + kVec<T> - 1) / kVec<T> + (kAligned ? 0 : 1);
      if (tokens * places > 152 * 2048) places = (places + kInFlight - 1) / kInFlight;
      const int lg = std::min(log2_up(places), 8);
      const int per = kMoveThreads >> lg;
      embed_kernel<T, IdT, kAligned>
          <<<static_cast<unsigned>((tokens + per - 1) / per), kMoveThreads, 0,
             static_cast<cudaStream_t>(stream)>>>(
              static_cast<const T*>(table), static_cast<int>(rows), static_cast<int>(width),
              table_stride, p, static_cast<int>(tokens), scale, static_cast<T*>(out), out_stride,
              lg);
      return launched();
    };
    const auto with_ids = [&](auto aligned) {
      return index_dtype == TBE_DT_I32 ? go(aligned, static_cast<const int32_t*>(ids))
                                       : go(aligned, static_cast<const int64_t*>(ids));
    };
    return vec ? with_ids(std::true_type{}) : with_ids(std::false_type{});
  });
}

extern "C" tbe_status tbe_embed_workspace_size(int64_t tokens, int64_t rows, int64_t width,
                                               size_t* bytes) {
  if (!bytes) return TBE_EINVAL;
  const tbe_status bad = check_sizes(tokens, rows, width);
  if (bad != TBE_OK) return bad;
  *bytes = static_cast<size_t>(layout_of(tokens, width).bytes);
  return TBE_OK;
}

extern "C" tbe_status tbe_embed_backward(const void* grad_out, int32_t dtype, int64_t tokens,
                                         int64_t width, int64_t grad_out_stride, const void* ids,
                                         int32_t index_dtype, int64_t rows, float scale,
                                         int32_t accumulate, void* grad_table, int32_t out_dtype,
                                         int64_t grad_table_stride, void* workspace,
                                         size_t ws_bytes, void* stream) {
  const tbe_status bad = check_sizes(tokens, rows, width);
  if (bad != TBE_OK) return bad;
  if (!dtype_bytes(dtype) || (out_dtype != dtype && out_dtype != TBE_DT_F32) ||
      (index_dtype != TBE_DT_I32 && index_dtype != TBE_DT_I64))
    return TBE_EUNSUPPORTED;
  if (!std::isfinite(scale)) return TBE_EINVAL;
  if (!rows || !width || (!tokens && accumulate)) return TBE_OK;
  const int b = dtype_bytes(dtype), ob = dtype_bytes(out_dtype);
  const Matrix in = {grad_out, grad_out_stride, b}, to = {grad_table, grad_table_stride, ob};
  if ((tokens && !in.good(tokens, width)) || !to.good(rows, width) ||
      !check_ids(ids, index_dtype, tokens))
    return TBE_EINVAL;
  const Layout l = layout_of(tokens, width);
  if (l.bytes && (!workspace || ws_bytes < static_cast<size_t>(l.bytes) ||
                  !aligned_to(workspace, 16)))
    return TBE_EWORKSPACE;
  const Bytes id_run = run_of(ids, tokens * (index_dtype == TBE_DT_I32 ? 4 : 8));
  const Bytes ws = run_of(l.bytes ? workspace : nullptr, l.bytes);
  const Bytes read = in.span(tokens, width), written = to.span(rows, width);
  if (overlap(written, read) || overlap(written, id_run) || overlap(written, ws) ||
      overlap(ws, read) || overlap(ws, id_run))
    return TBE_EINVAL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!tokens) return clear(grad_table, rows, width, grad_table_stride, ob, false, s);
  const bool vec = in.vectors(width, 16) && to.vectors(width, 16);
  const auto for_types = [&](auto f) {  // f(row type, result's type, aligned)
    return for_dtype(dtype, [&](auto t) {
      const auto with = [&](auto o) {
        return vec ? f(t, o, std::true_type{}) : f(t, o, std::false_type{});
      };
      return out_dtype == dtype ? with(t) : with(float{});
    });
  };
  if (tokens <= kFewTokens) {
    return for_types([&](auto t, auto o, auto aligned) {
      using T = decltype(t);
      using O = decltype(o);
      constexpr bool kAligned = decltype(aligned)::value;
      const int64_t places = (width + kVec<T> - 1) / kVec<T>;
      const int lg = std::min(log2_up(places), kFewLog), size = 1 << lg;
      const auto go = [&](auto* p) {
        using IdT = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
        FewArgs<IdT> few = {{grad_out, nullptr, grad_table, nullptr, grad_out_stride,
                             grad_table_stride, static_cast<int>(tokens), static_cast<int>(rows),
                             static_cast<int>(width), 0, 0, 0, scale, accumulate != 0},
                            p, 0};
        // about 64 KB a clearing CTA
        const int64_t slices = (places + size - 1) / size;
        few.range = static_cast<int>(std::clamp<int64_t>(65536 / (width * ob), 1, kFewRows));
        const int64_t ranges = accumulate ? 0 : (rows + few.range - 1) / few.range;
        const dim3 grid(static_cast<unsigned>(tokens + (ranges + slices - 1) / slices),
                        static_cast<unsigned>(slices));
        constexpr size_t kSums = kMoveThreads * kVec<T> * sizeof(float);
        return launch(embed_few_kernel<T, O, IdT, kAligned>, grid, kMoveThreads, kSums, kSums, false,
                      s, few, lg);
      };
      return index_dtype == TBE_DT_I32 ? go(static_cast<const int32_t*>(ids))
                                       : go(static_cast<const int64_t*>(ids));
    });
  }
  char* w = static_cast<char*>(workspace);
  SortPlan plan = plan_of(tokens, rows);
  plan.items[0] = reinterpret_cast<Item*>(w + l.items[0]);
  plan.items[1] = reinterpret_cast<Item*>(w + l.items[1]);
  const bool in_cluster = tokens <= (accumulate ? kOneLaunch : kOneCleared);
  const auto sort = [&](auto* p) {
    return in_cluster ? sort_in_cluster(p, plan, s)
                      : sort_in_grid(p, plan, reinterpret_cast<int*>(w + l.totals),
                                     reinterpret_cast<int*>(w + l.sums), s);
  };
  tbe_status st = index_dtype == TBE_DT_I32 ? sort(static_cast<const int32_t*>(ids))
                                            : sort(static_cast<const int64_t*>(ids));
  // The clearing runs beside the cluster, which leaves most of the GPU idle.
  if (st == TBE_OK && !accumulate)
    st = clear(grad_table, rows, width, grad_table_stride, ob, in_cluster, s);
  if (st != TBE_OK) return st;
  const int64_t piece = piece_of(tokens, width), pieces = (tokens + piece - 1) / piece;
  const int64_t slices = (width + 4 * kJoinLanes - 1) / (4 * kJoinLanes);
  // joining CTAs: four a multiprocessor (4097 tokens, 1000 columns: 18.7 us, with one 20.6, sixteen
  // 21.5; 52283 tokens of 2300 rows, 8 columns: 29.4, 34.6, 31.0)
  const int join =
      static_cast<int>(std::clamp<int64_t>(pieces * slices / (152 * 4), 1, kJoinPieces));
  const SumArgs args = {grad_out, plan.items[(plan.passes + 1) & 1], grad_table,
                        reinterpret_cast<float*>(w + l.parts), grad_out_stride, grad_table_stride,
                        static_cast<int>(tokens), static_cast<int>(rows), static_cast<int>(width),
                        static_cast<int>((width + 7) / 8 * 8), static_cast<int>(piece), join, scale,
                        accumulate != 0};
  return for_types([&](auto t, auto o, auto aligned) {
    using T = decltype(t);
    using O = decltype(o);
    constexpr bool kAligned = decltype(aligned)::value;
    const int64_t places = (width + kVec<T> - 1) / kVec<T>;
    const int lg = std::min(log2_up(places), 8);
    const int per = kMoveThreads >> lg;
    const dim3 grid(static_cast<unsigned>((pieces + per - 1) / per),
                    static_cast<unsigned>((places + (1 << lg) - 1) >> lg));
    constexpr size_t kRing = RowsAhead<T, kAligned>::kBytes * kMoveThreads;
    const size_t smem = kRing + ((per + 2) * piece + 2) * sizeof(Item);
    constexpr size_t kMostSmem = kRing + ((kMoveThreads + 2) * kMostPiece + 2) * sizeof(Item);
    const tbe_status summed = launch(embed_sum_kernel<T, O, kAligned>, grid, kMoveThreads, smem,
                                     kMostSmem, true, s, args, lg);
    if (summed != TBE_OK) return summed;
    const dim3 joins(static_cast<unsigned>((pieces + join - 1) / join),
                     static_cast<unsigned>(slices));
    return launch(embed_join_kernel<O>, joins, kJoinLanes * kJoinSegments, 0, 0, true, s, args);
  });
}
