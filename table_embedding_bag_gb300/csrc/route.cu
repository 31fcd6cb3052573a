// Routing: experts chosen for each token by score, bias and group, their weights, and
// the gradient of the weights in the logits.  The operations are specified in
// include/tbe_experts.h.
#include <cmath>
#include <type_traits>

#include "entry.cuh"
#include "tbe_experts.h"

namespace tbe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMostGroups = 32;  // a lane each
constexpr int kGroupRounds = 6;

struct RouteArgs {
  const void* logits;
  const float* bias;
  void* ids;
  float* weights;
  int64_t stride;
  int tokens, experts, k, groups, top_groups, group_best;
  float scale;
  bool sigmoid, renormalize, wide_ids;
  bool by_logits;  // no bias: the choices' order is that of the logits, which are compared
  // how a row's lanes share its experts: `group_lanes` = 2^log_lanes consecutive lanes a group of
  // `size` experts, `lane_experts` consecutive ones of them a lane
  int size, group_lanes, log_lanes, lane_experts;
  bool vectors;  // lane_experts is the kernel's V; all of a lane's experts exist and are aligned
};

constexpr float kClosed = -INFINITY;  // as a choice

// Choices in 64 bits in their order as integers: NaN above all, 0 for a closed expert is
// the caller's.
__device__ __forceinline__ unsigned long long order_of(double c) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(c + 0.0));
  if (c != c) return ~0ull;
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double value_of(unsigned long long o) {  // NaN of ~0
  return __longlong_as_double(static_cast<long long>(o >> 63 ? o & ~(1ull << 63) : ~o));
}

// Over the L lanes (a power of two) that share a row.  Maxima pass over NaN.
template <int L>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (L == 32) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
  }
}
template <int L, typename F>
__device__ __forceinline__ F row_sum(F v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// Whether a lane of this one's row says so.
template <int L>
__device__ __forceinline__ bool row_any(bool v) {
  const unsigned all = __ballot_sync(kAll, v);
  return (all >> (threadIdx.x & 31 & ~(L - 1)) & (kAll >> (32 - L))) != 0;
}

// What a row's scores need besides the logit: softmax's largest logit and sum.
struct RowScale {
  float top, sum;
};

// exp(x), off by 4 + 1.6 |x| units of 2^-24; 0 below 2^-126.
__device__ __forceinline__ float exp_near(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float reciprocal_near(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// `inverse`: one over softmax's sum.
__device__ __forceinline__ float score_of(float l, bool sigmoid, float top, float inverse) {
  return sigmoid ? reciprocal_near(1.f + exp_near(-l)) : exp_near(l - top) * inverse;
}

// Score and bias, the same wherever it is formed.
__device__ __forceinline__ float choice_of(float l, float b, bool sigmoid, float top,
                                           float inverse) {
  return sigmoid ? score_of(l, true, 0.f, 0.f) + b : fmaf(exp_near(l - top), inverse, b);
}

// A row's choice again in 64 bits, by the whole warp: few rows need it (see `step` below), but
// the last of them ends the launch.  room: the row's choices as integers in their order, 0 where
// an expert is closed.  Returns lane j's expert, -1 for none.
template <typename T>
__device__ __noinline__ int choose_exactly(const RouteArgs& P, const T* logits,
                                           unsigned long long* room) {
  const int lane = threadIdx.x & 31, size = P.size;
  double top = 0.0, sum = 1.0;
  if (!P.sigmoid) {
    float m = kClosed;
    for (int e = lane; e < P.experts; e += 32) m = fmaxf(m, to_f32(logits[e]));
    top = row_max<32>(m);
    sum = 0.0;
    for (int e = lane; e < P.experts; e += 32)
      sum += exp(static_cast<double>(to_f32(logits[e])) - top);
    sum = row_sum<32>(sum);
  }
  const auto score = [&](double l) {
    return P.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top) / sum;
  };
  for (int e = lane; e < P.experts; e += 32) {
    const double l = to_f32(logits[e]);
    const double c = P.by_logits || l == kClosed ? l : score(l) + P.bias[e];
    room[e] = c == kClosed ? 0 : order_of(c);
  }
  __syncwarp();
  if (P.groups > 1) {
    unsigned long long worth = 0;
    if (lane < P.groups) {
      unsigned long long first = 0, second = 0;
      for (int i = 0; i < size; ++i) {
        const unsigned long long o = room[lane * size + i];
        second = max(second, min(first, o));
        first = max(first, o);
      }
      if (first) {
        const bool two = P.group_best > 1;
        double w = value_of(first);
        if (two && P.by_logits) w = score(w);
        if (two && second) w += P.by_logits ? score(value_of(second)) : value_of(second);
        worth = order_of(w);
      }
    }
    int rank = 0;
    for (int g = 0; g < P.groups; ++g) {
      const unsigned long long o = __shfl_sync(kAll, worth, g);
      rank += o > worth || (o == worth && g < lane);
    }
    const unsigned open = __ballot_sync(kAll, worth != 0 && rank < P.top_groups);
    for (int g = 0; g < P.groups; ++g)
      if (!(open >> g & 1))
        for (int i = lane; i < size; i += 32) room[g * size + i] = 0;
    __syncwarp();
  }
  unsigned long long best = 0;  // this lane's largest
  int at = 0;
  const auto look = [&] {
    best = 0;
    for (int e = lane; e < P.experts; e += 32) {
      const unsigned long long o = room[e];
      if (o > best) best = o, at = e;
    }
  };
  look();
  int mine = -1;
  for (int r = 0; r < P.k; ++r) {
    // the largest, its upper and then its lower half, and of those alike the lowest expert
    const unsigned hi = __reduce_max_sync(kAll, static_cast<unsigned>(best >> 32));
    const bool in = best >> 32 == hi;
    const unsigned lo = __reduce_max_sync(kAll, in ? static_cast<unsigned>(best) : 0u);
    if (!hi) break;  // an open choice has bits there
    const bool tied = in && static_cast<unsigned>(best) == lo;
    const int e = static_cast<int>(__reduce_min_sync(kAll, tied ? at : INT32_MAX));
    if (lane == r) mine = e;
    if (tied && at == e) {
      room[e] = 0;
      look();
    }
  }
  __syncwarp();
  return mine;
}

// Whether a row of L lanes has an expert whose choice may be the one of logit l and bias b, which
// is `last`, without being the same logit and bias.  by: what the errors of both come to at most.
template <typename T, int L>
__device__ __noinline__ bool others_near(const RouteArgs& P, const T* logits, float l, float b,
                                         float last, float by, float top, float inverse) {
  bool found = false;
  for (int e = threadIdx.x & (L - 1); e < P.experts; e += L) {
    const float le = to_f32(logits[e]), be = P.bias[e];
    const float s = le == kClosed ? kClosed : choice_of(le, be, P.sigmoid, top, inverse);
    found |= s != kClosed && !(le == l && be == b) &&
             !(fabsf(last - s) > by + 0x1p-23f * fmaxf(fabsf(last), fabsf(s)));
  }
  return row_any<L>(found);
}

// The candidates of rows of L lanes, lane j with expert `mine` (-1: none) of logit l and bias b,
// put in the order of their sigmoid choices in 64 bits.  room: 32 entries.
template <int L>
__device__ __noinline__ int order_exactly(int mine, float l, float b, int* room) {
  const int lane = threadIdx.x & 31, first = lane & ~(L - 1);
  const double c = mine >= 0 ? 1.0 / (1.0 + exp(-static_cast<double>(l))) + b : kClosed;
  room[lane] = -1;  // should ranks collide, which NaN alone could do, no entry is left unset
  __syncwarp();
  int rank = 0;
  for (int j = 0; j < L; ++j) {
    const double other = __shfl_sync(kAll, c, first + j);
    const int e = __shfl_sync(kAll, mine, first + j);
    // those that are none keep their places at the end
    rank += other > c || (other == c && (mine >= 0 ? e >= 0 && e < mine : first + j < lane));
  }
  __syncwarp();
  room[first + rank] = mine;
  __syncwarp();
  mine = room[lane];
  __syncwarp();
  return mine;
}

// sigmoid(x), to fp32's end at both sides.
__device__ __forceinline__ float logistic(float x) {
  const float e = expf(-fabsf(x));
  return __fdiv_rn(x < 0.f ? e : 1.f, 1.f + e);
}

// Weights of the chosen, before the scale: lane j of a row has the j-th expert's logit, `on`
// where there is one.  By expf and rounded divisions, in both directions: an expert is chosen by
// approximate scores only where their errors do not matter, but its weight is a result.
template <int L>
__device__ __forceinline__ float weight_of(float l, bool on, bool sigmoid, bool renormalize,
                                           RowScale r) {
  if (!renormalize) {
    if (!on) return 0.f;
    return sigmoid ? logistic(l) : __fdiv_rn(expf(l - r.top), r.sum);
  }
  const float top = row_max<L>(on ? l : kClosed);
  // sigmoid(l) is exp(l) to a quarter of the last bit where no logit is above -18, and exp(l - top)
  // does not underflow
  const float p = !on ? 0.f : sigmoid && !(top < -18.f) ? logistic(l) : expf(l - top);
  const float sum = row_sum<L>(p);
  if (!on) return 0.f;
  // a NaN among the row's scores makes every softmax weight one
  return !sigmoid && r.sum != r.sum ? r.sum : __fdiv_rn(p, sum);
}

// The K experts with the largest choices, in their order: lane j of a row gets the j-th (-1 for
// none).  Takes what it has chosen out of c.  One expert a round.
template <int V, int L>
__device__ __forceinline__ int choose_in_rounds(float (&c)[V], int e0, int K) {
  const int lane = threadIdx.x & 31, first = lane & ~(L - 1), place = lane & (L - 1);
  float most = c[0];
#pragma unroll
  for (int v = 1; v < V; ++v) most = fmaxf(most, c[v]);
  int mine = -1;
  for (int r = 0; r < K; ++r) {
    const float best = row_max<L>(most);
    const unsigned who = __ballot_sync(kAll, most == best && best != kClosed);
    if (!who) break;
    const unsigned row = who >> first & (kAll >> (32 - L));
    const int winner = row ? __ffs(row) - 1 : -1;
    int at = 0;
    if (place == winner) {
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (c[v] == best) at = v;
      most = kClosed;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (v == at) c[v] = kClosed;
        most = fmaxf(most, c[v]);
      }
      at += e0;
    }
    at = __shfl_sync(kAll, at, first + (row ? winner : 0));
    if (place == r && row) mine = at;
  }
  return mine;
}

// A warp's shared memory, in doubles: a row's choices in 64 bits, or candidates (read in 16
// bytes).
__host__ __device__ constexpr int room_of(int experts) { return (experts + 33) & ~1; }

// Room for candidates.
struct Candidates {
  float c[32];
  int e[32];
};

// Chosen ones up to which rows of L lanes have few enough candidates (of normally distributed choices
// one row in 30 has more than 16 with 9 of 128 experts, one in 100 more than 8 with 4 of 64).
__host__ __device__ constexpr int most_by_bound(int L) { return L == 32 ? 16 : L == 16 ? 9 : 4; }

// The same with several experts a lane.  The K-th largest of the lanes' largest choices bounds the
// K-th choice from below, so only choices from there on are candidates, a few more than K;
// they are moved to shared memory, ranked against one another, a lane each, and put in
// order: lane j of a row gets the j-th, past K too.  In rounds every expert chosen costs a look
// over the lane's V choices (65536 rows of bf16, 8 of 128: 21.6 us, in rounds 31.8; 4 of 64: 10.4 and
// 11.6; 8 of 256 by sigmoid and bias, fp32: 43.9 and 77).  *bound: no other choice is above it.
// -2 throughout where a row has more candidates than lanes.
template <int V, int L>
__device__ __forceinline__ int choose_by_bound(float (&c)[V], int e0, int K, Candidates& room,
                                               float* bound) {
  const int lane = threadIdx.x & 31, place = lane & (L - 1), row = lane & ~(L - 1);
  float left = c[0];
#pragma unroll
  for (int v = 1; v < V; ++v) left = fmaxf(left, c[v]);
  float least = kClosed;
  if constexpr (L == 32) {
#pragma unroll 4
    for (int r = 0; r < K; ++r) {
      least = row_max<L>(left);
      if (left == least) left = kClosed;
    }
  } else {  // the least of those that fewer than K are above
    int above = 0;
#pragma unroll
    for (int o = 1; o < L; ++o) above += __shfl_xor_sync(kAll, left, o) > left;
    least = -row_max<L>(above < K ? -left : kClosed);
  }
  *bound = least;
  if (least == kClosed) least = -3.402823466e38f;  // open ones only
  int count = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) count += c[v] >= least;
  int upto = count;
#pragma unroll
  for (int o = 1; o < L; o <<= 1) {
    const int y = __shfl_up_sync(kAll, upto, o);
    if (place >= o) upto += y;
  }
  const int all = __shfl_sync(kAll, upto, row + L - 1);
  const bool many = L == 32 ? all > L : __any_sync(kAll, all > L);
  if (many) return -2;  // many alike, or few lanes open
  room.c[lane] = kClosed;
  __syncwarp();
  int at = row + upto - count;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (c[v] >= least) {
      room.c[at] = c[v];
      room.e[at++] = e0 + v;
    }
  __syncwarp();
  const float mine = room.c[lane];
  const int e = place < all ? room.e[lane] : -1;
  int rank = 0;
  for (int j = 0; j < (L == 32 ? all : L); j += 4) {
    const float4 o = *reinterpret_cast<const float4*>(room.c + row + j);
    rank += o.x > mine;
    rank += o.y > mine;
    rank += o.z > mine;
    rank += o.w > mine;
  }
  // Choices that are alike share a rank, and the ranks' sum falls short: they take the order of
  // the experts, in which they stand.
  const int ranks = all * (all - 1) / 2;  // of a row without
  const int short_of = L == 32 ? 0 : place == 0 ? ranks : 0;
  if (static_cast<int>(__reduce_add_sync(kAll, (place < all ? rank : 0) - short_of)) !=
      (L == 32 ? ranks : 0))
    for (int j = 0; j < all; ++j) rank += room.c[row + j] == mine && j < place;
  __syncwarp();
  if (place < all) room.e[row + rank] = e;
  __syncwarp();
  const int sorted = place < all ? room.e[lane] : -1;
  __syncwarp();
  return sorted;
}

// A row's experts are shared by L lanes, V consecutive ones a lane at most; 32 / L rows a warp.
//
// Instructions bound it (65536 rows, eight of 256 experts in four of eight groups by sigmoid and
// bias: 53 us for a floor of 10.5 in bytes; 769 a row, issued in 85 % of the cycles), so reductions
// are the warp's own (redux), the choice looks over few candidates, and what exact arithmetic
// would cost is kept for the rows that need it.  Five CTAs a multiprocessor: 53.6 us, with four
// 56.5, with six 55.6; in sixteen other forms, of 8 to 32 lanes a row, five are within 5 % of the best
// of the three, though at 48 registers those of 8 and 16 lanes spill 36 to 68 bytes.
// kCandidates: choose_by_bound, which has a kernel of its own as its registers cost the rounds 5 %.
template <typename T, int V, int L, bool kCandidates>
__global__ void __launch_bounds__(256, V <= 8 ? 5 : 1)
    route_kernel(const __grid_constant__ RouteArgs P) {
  constexpr int kRows = 32 / L;
  extern __shared__ __align__(16) double route_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, place = lane & (L - 1);
  const int64_t token0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp) * kRows;
  if (token0 >= P.tokens) return;
  const int64_t token = token0 + lane / L;
  const bool live = token < P.tokens;
  const T* logits = static_cast<const T*>(P.logits) + (live ? token : token0) * P.stride;
  double* room = route_smem + warp * room_of(P.experts);

  // this lane's experts: e0 .. e0 + mine - 1, of its group
  const int size = P.size, group = place >> P.log_lanes;
  const int in_group = (place & (P.group_lanes - 1)) * P.lane_experts;
  const int e0 = group * size + in_group;
  int count = size - in_group < P.lane_experts ? size - in_group : P.lane_experts;
  if (!live || group >= P.groups) count = 0;
  float c[V];
  {
    constexpr int kPart = V * sizeof(T) < 16 ? V : 16 / static_cast<int>(sizeof(T));
    if (P.vectors && count > 0) {
#pragma unroll
      for (int v = 0; v < V; v += kPart) {
        const Pack<T, kPart> p = *reinterpret_cast<const Pack<T, kPart>*>(logits + e0 + v);
#pragma unroll
        for (int i = 0; i < kPart; ++i) c[v + i] = to_f32(p.v[i]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = v < count ? to_f32(logits[e0 + v]) : kClosed;
    }
  }

  RowScale scale = {0.f, 1.f};
  float inverse = 1.f;
  const bool by_score = !P.by_logits || (P.groups > 1 && P.group_best > 1);
  if (!P.sigmoid && (by_score || !P.renormalize)) {
    float top = c[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, c[v]);
    scale.top = row_max<L>(top);
    float part[V];
#pragma unroll
    for (int v = 0; v < V; ++v)  // of weights, not only of choices, where they are not renormalised
      part[v] = P.renormalize ? exp_near(c[v] - scale.top) : expf(c[v] - scale.top);
#pragma unroll
    for (int o = V / 2; o; o >>= 1)
#pragma unroll
      for (int v = 0; v < o; ++v) part[v] += part[v + o];
    scale.sum = row_sum<L>(part[0]);
    inverse = reciprocal_near(scale.sum);
  }

  // from logits to choices
  if (!P.by_logits) {
    float b[V];
    constexpr int kPart = V < 4 ? V : 4;
    if (P.vectors && count > 0) {
#pragma unroll
      for (int v = 0; v < V; v += kPart) {
        const Pack<float, kPart> p = *reinterpret_cast<const Pack<float, kPart>*>(P.bias + e0 + v);
#pragma unroll
        for (int i = 0; i < kPart; ++i) b[v + i] = p.v[i];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] = v < count ? P.bias[e0 + v] : 0.f;
    }
    if (P.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        c[v] = c[v] == kClosed ? kClosed : choice_of(c[v], b[v], true, 0.f, 0.f);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        c[v] = c[v] == kClosed ? kClosed : choice_of(c[v], b[v], false, scale.top, inverse);
    }
  }
  // NaN, or infinities of both signs
  float all = c[0];
#pragma unroll
  for (int v = 1; v < V; ++v) all += c[v];
  const bool odd = (scale.sum != scale.sum && scale.top != kClosed) || (all != all && count > 0);

  // Two choices closer than their errors may be the other way round in exact arithmetic.  In units
  // of 2^-24, a sigmoid score is off by at most 4.2 (the exponential's 4 + 1.6 |l| times
  // s (1 - s), 1.1 at most, the sum's 1 and the reciprocal's 2), a softmax score x below the
  // row's top by 34 + 2 |x| times itself (exponential 4 + 2 |x|, the sum's terms 4 + 2 mean |x|,
  // where that mean is at most log 1024, its ten additions, reciprocal and product), and so by
  // 35 times the row's largest; its sum with the bias by one unit of itself.  step: twice the
  // bound that holds for every expert.
  const float step = P.sigmoid ? 0x1.1p-21f : 0x1.2p-18f * inverse;
  bool unsure = row_any<L>(odd), near = false;

  if (P.groups > 1) {
    float first = kClosed, second = kClosed;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      second = fmaxf(second, fminf(first, c[v]));
      first = fmaxf(first, c[v]);
    }
    for (int o = P.group_lanes >> 1; o; o >>= 1) {
      const float f = __shfl_xor_sync(kAll, first, o), s = __shfl_xor_sync(kAll, second, o);
      second = fmaxf(fmaxf(second, s), fminf(first, f));
      first = fmaxf(first, f);
    }
    float worth = first, size_of = first == kClosed ? 0.f : fabsf(first);  // of what it sums
    if (P.group_best > 1 && first != kClosed) {
      if (P.by_logits) {
        first = score_of(first, P.sigmoid, scale.top, inverse);
        if (second != kClosed) second = score_of(second, P.sigmoid, scale.top, inverse);
      }
      worth = second != kClosed ? first + second : first;
      size_of = second != kClosed ? fabsf(first) + fabsf(second) : fabsf(first);
    }
    // The groups worth most, one a round where a round is one reduction (eight instructions,
    // ranking takes nine for every other group); where two are worth the same, by their ranks.
    bool open = false, ranked = L < 32 || P.top_groups > kGroupRounds;
    float last = kClosed, next = kClosed;  // the least worth that is taken, the largest left
    if (!ranked) {
      float left = worth;
      for (int r = 0; r < P.top_groups && !ranked; ++r) {
        const float best = row_max<L>(left);
        const bool mine = left == best && best != kClosed;
        ranked = __popc(__ballot_sync(kAll, mine)) > P.group_lanes;
        if (mine) left = kClosed, open = true;
        if (best != kClosed) last = best;
      }
      next = row_max<L>(left);
    }
    if (ranked) {
      int rank = 0;
#pragma unroll 2
      for (int o = P.group_lanes; o < L; o += P.group_lanes) {
        const float other = __shfl_xor_sync(kAll, worth, o);
        rank += other > worth || (other == worth && (place ^ o) < place);
      }
      open = worth != kClosed && rank < P.top_groups;
      last = -row_max<L>(open ? -worth : kClosed);
      next = row_max<L>(!open ? worth : kClosed);
    }
    if (by_score) {
      const float largest = row_max<L>(size_of);
      // two sums of two choices, each rounded, and rounded themselves
      unsure |= next != kClosed && !(last - next > 2.f * step + 0x1p-22f * largest);
    }
    if (!open) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = kClosed;
    }
  }

  const int K = P.by_logits ? P.k : P.k + 1;
  int mine = -2;  // lane j of the row: the j-th expert
  float bound = kClosed;
  if constexpr (kCandidates)
    mine = choose_by_bound<V, L>(c, e0, K, *reinterpret_cast<Candidates*>(room), &bound);
  const bool in_rounds = mine == -2;
  if (in_rounds) mine = choose_in_rounds<V, L>(c, e0, K);
  float chosen = mine >= 0 ? to_f32(logits[mine]) : 0.f;
  if (!P.by_logits) {
    // neighbours in the order that fp32 does not tell apart; the same logit and bias tie in any
    // arithmetic
    const float b = mine >= 0 ? P.bias[mine] : 0.f;
    const float score = mine >= 0 ? score_of(chosen, P.sigmoid, scale.top, inverse) : 0.f;
    const float s = mine >= 0 ? choice_of(chosen, b, P.sigmoid, scale.top, inverse) : kClosed;
    // (softmax: and by what the exponential drops below 2^-126)
    const float below = scale.top - chosen;
    const float off =
        P.sigmoid ? 0x1.1p-22f : fmaf(score * 0x1p-24f, 34.f + 2.f * below, 0x1p-125f);
    const float lp = __shfl_up_sync(kAll, chosen, 1), bp = __shfl_up_sync(kAll, b, 1);
    const float sp = __shfl_up_sync(kAll, s, 1), op = __shfl_up_sync(kAll, off, 1);
    const auto far = [&](float more, float less, float by) {
      return more - less > by + 0x1p-23f * fmaxf(fabsf(less), fabsf(more));
    };
    // The one past the last that is taken stands for all that are left, which are no larger here
    // but may be off by more than it is: by half a step at most.
    const float by = place == P.k ? op + 0.5f * step : op + off;
    const bool close = place > 0 && place < K && mine >= 0 && !far(sp, s, by);
    const bool alike = lp == chosen && bp == b;
    near = row_any<L>(close && !alike) && !unsure;
    // Where the last that is taken and the one past it are alike, that one does not stand for those
    // behind it.
    const bool hidden = close && alike && place == P.k;
    if (__any_sync(kAll, hidden)) {
      const int edge = (lane & ~(L - 1)) + P.k;
      const float l = __shfl_sync(kAll, chosen, edge), bias = __shfl_sync(kAll, b, edge);
      const float last = __shfl_sync(kAll, s, edge), width = __shfl_sync(kAll, by, edge);
      const bool others = others_near<T, L>(P, logits, l, bias, last, width, scale.top, inverse);
      near |= row_any<L>(hidden) && others && !unsure;
    }
    if (__any_sync(kAll, near)) {
      // the candidates suffice where the last that is taken is above all others for certain
      const int edge = (lane & ~(L - 1)) + P.k - 1;
      const float last = __shfl_sync(kAll, s, edge);
      const float next = in_rounds ? __shfl_sync(kAll, s, edge + 1 < 32 ? edge + 1 : 31) : bound;
      const bool enough = P.sigmoid && (next == kClosed || far(last, next, step));
      const int sorted = order_exactly<L>(mine, chosen, b, reinterpret_cast<int*>(room));
      if (near && enough) {
        mine = sorted;
        chosen = mine >= 0 ? to_f32(logits[mine]) : 0.f;
      } else {
        unsure |= near;
      }
    }
  }
  const unsigned again = __ballot_sync(kAll, unsure);
  if (again) {
#pragma unroll 1
    for (int r = 0; r < kRows; ++r) {
      if (!(again >> (r * L) & 1)) continue;
      const int64_t t = token0 + r < P.tokens ? token0 + r : token0;
      const int found = choose_exactly(P, static_cast<const T*>(P.logits) + t * P.stride,
                                       reinterpret_cast<unsigned long long*>(room));
      const int my = __shfl_sync(kAll, found, place);
      if (lane / L == r) mine = my;
    }
    chosen = mine >= 0 ? to_f32(logits[mine]) : 0.f;
  }
  if (place >= P.k) mine = -1;  // the one past the last
  const float w = weight_of<L>(chosen, mine >= 0, P.sigmoid, P.renormalize, scale);
  if (place < P.k && live) {
    const int64_t at = token * P.k + place;
    if (P.wide_ids) static_cast<int64_t*>(P.ids)[at] = mine;
    else static_cast<int*>(P.ids)[at] = mine;
    P.weights[at] = mine >= 0 ? P.scale * w : 0.f;
  }
}

struct RouteGradArgs {
  const float* grad_weights;
  const void *logits, *ids;
  void* grad;
  int64_t stride, grad_stride;
  int tokens, experts, k;
  float scale;
  bool sigmoid, renormalize, wide_ids;
  bool vectors;  // the rows of grad allow 16-byte stores from end to end
};

// L lanes a token, lane j for its j-th expert.  Most of a row does not depend on what is
// read, so it is written at once, and the chosen experts' gradients follow over it: the loads'
// and sums' latencies pass while the stores are on their way.  65536 x 256 fp32, eight chosen:
// 19 us, 5.5 TB/s of what moves: each logit read brings its sector of 32 bytes.
template <typename T, int L>
__global__ void __launch_bounds__(256)
    route_backward_kernel(const __grid_constant__ RouteGradArgs P) {
  constexpr int V = kVec<T>;
  const int lane = threadIdx.x & 31, place = lane & (L - 1);
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (256 / L) + threadIdx.x / L;
  const bool live = token < P.tokens;  // the others take part in the sums
  const T* logits = static_cast<const T*>(P.logits) + (live ? token : 0) * P.stride;
  T* grad = static_cast<T*>(P.grad) + (live ? token : 0) * P.grad_stride;
  const int experts = live ? P.experts : 0;
  const bool whole = !P.sigmoid && !P.renormalize;  // every logit has a gradient
  // value(i): the gradient of expert i's logit were it not chosen
  const auto fill = [&](auto value) {
    if (P.vectors) {
      for (int i = place * V; i < experts; i += L * V) {
        float f[V];
#pragma unroll
        for (int u = 0; u < V; ++u) f[u] = value(i + u);
        store_vec(grad + i, from_floats<T>(f));
      }
    } else {
      for (int i = place; i < experts; i += L) grad[i] = from_f32<T>(value(i));
    }
  };
  if (!whole) fill([](int) { return 0.f; });
  int64_t id = -1;
  if (live && place < P.k) {
    const int64_t at = token * P.k + place;
    id = P.wide_ids ? static_cast<const int64_t*>(P.ids)[at] : static_cast<const int*>(P.ids)[at];
  }
  const bool on = id >= 0 && id < experts;
  const int e = on ? static_cast<int>(id) : -1;
  const float l = on ? to_f32(logits[e]) : 0.f;
  const float g = on ? P.scale * P.grad_weights[token * P.k + place] : 0.f;
  RowScale scale = {0.f, 1.f};
  if (whole) {
    float top = kClosed;
    for (int i = place; i < experts; i += L) top = fmaxf(top, to_f32(logits[i]));
    scale.top = row_max<L>(top);
    float sum = 0.f;
    for (int i = place; i < experts; i += L) sum += expf(to_f32(logits[i]) - scale.top);
    scale.sum = row_sum<L>(sum);
  }
  const float p = weight_of<L>(l, on, P.sigmoid, P.renormalize, scale);
  const float mean = P.sigmoid && !P.renormalize ? 0.f : row_sum<L>(g * p);
  if (whole)
    fill([&](int i) {  // zeros where every expert is closed
      return scale.top == kClosed
                 ? 0.f
                 : __fdiv_rn(expf(to_f32(logits[i]) - scale.top), scale.sum) * -mean;
    });
  // where an expert is named more than once, the first lane that does adds up the others' in
  // their order; softmax's mean counts once
  const unsigned same = __match_any_sync(kAll, on ? (lane & ~(L - 1)) << 16 | e : -1 - lane);
  const bool first = (same & ((1u << lane) - 1)) == 0;
  float of_score = g;
  if (__any_sync(kAll, !first)) {
    of_score = 0.f;
    for (int j = 0; j < 32; ++j) {
      const float v = __shfl_sync(kAll, g, j);
      if (same >> j & 1) of_score += v;
    }
  }
  float d;
  if (whole) {
    d = p * (of_score - mean);
  } else {
    // as many times the mean as the expert is named
    d = p * (of_score - static_cast<float>(__popc(same)) * mean);
    if (P.sigmoid) d *= logistic(-l);  // 1 - sigmoid(l)
  }
  __syncwarp();
  if (on && first) grad[e] = from_f32<T>(d);
}

// -------------------------------------------------------------- host

tbe_status check_route(int32_t dtype, int64_t tokens, int32_t experts, int32_t score, int32_t k,
                       int32_t index_dtype, float scale) {
  if (tokens < 0 || experts < 1 || k < 1) return TBE_EINVAL;
  if (score != TBE_SCORE_SOFTMAX && score != TBE_SCORE_SIGMOID) return TBE_EINVAL;
  if (!std::isfinite(scale)) return TBE_EINVAL;
  if (!dtype_bytes(dtype) || (index_dtype != TBE_DT_I32 && index_dtype != TBE_DT_I64) ||
      experts > TBE_MAX_EXPERTS || k > TBE_MAX_CHOSEN || tokens > INT32_MAX / k)
    return TBE_EUNSUPPORTED;
  return TBE_OK;
}

int id_bytes(int32_t index_dtype) { return index_dtype == TBE_DT_I32 ? 4 : 8; }

// How rows are shared: as few lanes as hold the chosen ones (and the next) with at most eight
// experts each, so that a warp's reductions serve several rows; but a warp a row where that makes
// the candidates few (65536 rows: 10 of 128 31 us and 39, 12 32 and 44; sixteen lanes a row for the
// same reason are slower, 6 of 64 17.3 and 14.7).
template <typename T>
tbe_status launch_route(RouteArgs args, cudaStream_t s) {
  const int size = args.experts / args.groups;
  int slots = 1;  // groups, rounded up to a power of two
  while (slots < args.groups) slots *= 2;
  int lanes = 8;
  const int kept = args.by_logits ? args.k : args.k + 1;
  const auto each = [&](int l) {  // experts of a lane, of l a row
    return l < slots ? INT32_MAX : (size + l / slots - 1) / (l / slots);
  };
  while (lanes < 32 && (lanes < kept || each(lanes) > 8 ||
                        (lanes == 16 && kept > most_by_bound(16) && each(32) > 2)))
    lanes *= 2;
  args.size = size;
  args.group_lanes = lanes / slots;
  for (args.log_lanes = 0; 1 << args.log_lanes < args.group_lanes;) ++args.log_lanes;
  args.lane_experts = each(lanes);
  const auto go = [&](auto v, auto l) {
    constexpr int V = decltype(v)::value, L = decltype(l)::value;
    constexpr int kPart = V * sizeof(T) < 16 ? V : 16 / static_cast<int>(sizeof(T));
    args.vectors = args.lane_experts == V && size % V == 0 && args.stride % kPart == 0 &&
                   aligned_to(args.logits, kPart * sizeof(T)) && aligned_to(args.bias, 16);
    const int warps = args.experts > 512 ? 4 : 8, rows = warps * (32 / L);
    const auto run = [&](auto candidates) {
      route_kernel<T, V, L, decltype(candidates)::value>
          <<<static_cast<unsigned>((args.tokens + int64_t(rows) - 1) / rows), warps * 32,
             warps * room_of(args.experts) * sizeof(double), s>>>(args);
      return launched();
    };
    if constexpr (V >= 4) {
      if (kept <= most_by_bound(L)) return run(std::true_type{});
    }
    return run(std::false_type{});
  };
  const auto with = [&](auto l) {
    constexpr int L = decltype(l)::value;
    if (args.lane_experts <= 2) return go(std::integral_constant<int, 2>{}, l);
    if (args.lane_experts <= 4) return go(std::integral_constant<int, 4>{}, l);
    if (L < 32 || args.lane_experts <= 8) return go(std::integral_constant<int, 8>{}, l);
    if constexpr (L == 32) {
      if (args.lane_experts <= 16) return go(std::integral_constant<int, 16>{}, l);
      if (args.lane_experts <= 32) return go(std::integral_constant<int, 32>{}, l);
      return go(std::integral_constant<int, 64>{}, l);  // groups that leave lanes idle
    }
    return TBE_EUNSUPPORTED;
  };
  if (lanes == 8) return with(std::integral_constant<int, 8>{});
  if (lanes == 16) return with(std::integral_constant<int, 16>{});
  return with(std::integral_constant<int, 32>{});
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_expert_route(const void* logits, int32_t dtype, int64_t tokens,
                                       int32_t experts, int64_t logits_stride, const float* bias,
                                       int32_t score, int32_t k, int32_t groups,
                                       int32_t top_groups, int32_t group_best,
                                       int32_t renormalize, float scale, void* ids,
                                       int32_t index_dtype, float* weights, void* stream) {
  const tbe_status bad = check_route(dtype, tokens, experts, score, k, index_dtype, scale);
  if (bad != TBE_OK) return bad;
  if (groups < 1 || experts % groups || top_groups < 1 || top_groups > groups || group_best < 1 ||
      group_best > 2 || k > top_groups * (experts / groups))
    return TBE_EINVAL;
  if (groups > kMostGroups) return TBE_EUNSUPPORTED;
  if (!tokens) return TBE_OK;
  const Matrix in = {logits, logits_stride, dtype_bytes(dtype)};
  if (!in.good(tokens, experts) || !ids || !aligned_to(ids, id_bytes(index_dtype)) || !weights ||
      !aligned_to(weights, 4) || !aligned_to(bias, 4))
    return TBE_EINVAL;
  const Bytes written[2] = {run_of(ids, tokens * k * id_bytes(index_dtype)),
                            run_of(weights, tokens * k * 4)};
  const Bytes read[2] = {in.span(tokens, experts), run_of(bias, bias ? int64_t(experts) * 4 : 0)};
  for (const Bytes& w : written)
    for (const Bytes& r : read)
      if (overlap(w, r)) return TBE_EINVAL;
  if (overlap(written[0], written[1])) return TBE_EINVAL;
  const RouteArgs args = {logits, bias, ids, weights, logits_stride, static_cast<int>(tokens),
                          experts, k, groups, top_groups, group_best, scale,
                          score == TBE_SCORE_SIGMOID, renormalize != 0, index_dtype == TBE_DT_I64,
                          !bias, 0, 0, 0, 0, false};
  return for_dtype(dtype, [&](auto t) {
    return launch_route<decltype(t)>(args, static_cast<cudaStream_t>(stream));
  });
}

extern "C" tbe_status tbe_expert_route_backward(const float* grad_weights, const void* logits,
                                                int32_t dtype, int64_t tokens, int32_t experts,
                                                int64_t logits_stride, const void* ids,
                                                int32_t index_dtype, int32_t k, int32_t score,
                                                int32_t renormalize, float scale,
                                                void* grad_logits, int64_t grad_stride,
                                                void* stream) {
  const tbe_status bad = check_route(dtype, tokens, experts, score, k, index_dtype, scale);
  if (bad != TBE_OK) return bad;
  if (!tokens) return TBE_OK;
  const int b = dtype_bytes(dtype);
  const Matrix in = {logits, logits_stride, b}, out = {grad_logits, grad_stride, b};
  if (!in.good(tokens, experts) || !out.good(tokens, experts) || !ids ||
      !aligned_to(ids, id_bytes(index_dtype)) || !grad_weights || !aligned_to(grad_weights, 4))
    return TBE_EINVAL;
  const Bytes written = out.span(tokens, experts);
  if (overlap(written, in.span(tokens, experts)) ||
      overlap(written, run_of(ids, tokens * k * id_bytes(index_dtype))) ||
      overlap(written, run_of(grad_weights, tokens * k * 4)))
    return TBE_EINVAL;
  const RouteGradArgs args = {grad_weights, logits, ids, grad_logits, logits_stride, grad_stride,
                              static_cast<int>(tokens), experts, k, scale,
                              score == TBE_SCORE_SIGMOID, renormalize != 0,
                              index_dtype == TBE_DT_I64, out.vectors(experts, 16)};
  return for_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const auto go = [&](auto lanes) {
      constexpr int L = decltype(lanes)::value, kRows = 256 / L;
      route_backward_kernel<T, L>
          <<<static_cast<unsigned>((tokens + kRows - 1) / kRows), 256, 0,
             static_cast<cudaStream_t>(stream)>>>(args);
      return launched();
    };
    if (k <= 8) return go(std::integral_constant<int, 8>{});
    if (k <= 16) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
  });
}
