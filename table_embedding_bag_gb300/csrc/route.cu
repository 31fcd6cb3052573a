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

struct RouteArgs {
  const void* logits;
  const float* bias;
  void* ids;
  float* weights;
  int64_t stride;
  int tokens, experts, k, groups, top_groups, group_best;
  float scale;
  bool sigmoid, renormalize, wide_ids;
  bool by_logits;  // the choices' order is that of the logits
};

// Values in their order as integers: 0 for an expert that is closed, NaN above all.
__device__ __forceinline__ uint32_t order_of(float c) {
  const uint32_t b = __float_as_uint(c + 0.f);  // -0 is 0
  if (c != c) return 0xffffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long order_of(double c) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(c + 0.0));
  if (c != c) return ~0ull;
  return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// What a row's scores need besides the logit: softmax's largest logit and sum.
struct RowScale {
  float top, sum;
};

__device__ __forceinline__ float score_of(float l, bool sigmoid, RowScale r) {
  return sigmoid ? __fdividef(1.f, 1.f + __expf(-l)) : __fdividef(__expf(l - r.top), r.sum);
}

// The groups (a bit each) that are worth most: lane g holds group g's worth as an integer in
// order, 0 where no expert of it is open.
template <typename Order>
__device__ __forceinline__ unsigned best_groups(Order mine, int groups, int top) {
  const int lane = threadIdx.x & 31;
  int rank = 0;
  for (int g = 0; g < groups; ++g) {
    const Order o = __shfl_sync(kAll, mine, g);
    rank += o > mine || (o == mine && g < lane);
  }
  return __ballot_sync(kAll, lane < groups && mine != 0 && rank < top);
}

// The choice again in 64 bits, without a thought for speed: some rows in a thousand need it.
// c: room for the row's choices.  Returns lane j's expert, -1 for none.
template <typename T>
__device__ __noinline__ int choose_exactly(const RouteArgs& P, const T* logits, double* c) {
  const int lane = threadIdx.x & 31, size = P.experts / P.groups;
  const double closed = -INFINITY;
  double top = closed, sum = 0.0;
  if (!P.sigmoid) {
    float m = -INFINITY;
    for (int e = lane; e < P.experts; e += 32) m = fmaxf(m, to_f32(logits[e]));
    top = warp_max(m);
    for (int e = lane; e < P.experts; e += 32)
      sum += exp(static_cast<double>(to_f32(logits[e])) - top);
    sum = warp_sum(sum);
  }
  for (int e = lane; e < P.experts; e += 32) {
    const double l = to_f32(logits[e]);
    double v = P.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top) / sum;
    if (P.bias) v += P.bias[e];
    c[e] = l == closed ? closed : v;
  }
  __syncwarp();
  unsigned open = kAll;
  if (P.groups > 1) {
    unsigned long long worth = 0;
    if (lane < P.groups) {
      double first = closed, second = closed;
      for (int i = 0; i < size; ++i) {
        const double v = c[lane * size + i];
        if (order_of(v) > order_of(first)) second = first, first = v;
        else if (order_of(v) > order_of(second)) second = v;
      }
      if (first != closed)
        worth = order_of(P.group_best > 1 && second != closed ? first + second : first);
    }
    open = best_groups(worth, P.groups, P.top_groups);
  }
  int mine = -1;
  for (int r = 0; r < P.k; ++r) {
    unsigned long long best = 0;
    int at = 0;
    for (int e = lane; e < P.experts; e += 32) {
      const double v = c[e];
      const unsigned long long o = v == closed || !(open >> (e / size) & 1) ? 0 : order_of(v);
      if (o > best) best = o, at = e;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(kAll, best, o);
      const int where = __shfl_xor_sync(kAll, at, o);
      if (other > best || (other == best && where < at)) best = other, at = where;
    }
    if (!best) break;
    if (lane == r) mine = at;
    __syncwarp();
    if (lane == 0) c[at] = closed;
    __syncwarp();
  }
  return mine;
}

// Weights of the chosen, before the scale: lane j has expert j's logit, `on` where there is one.
__device__ __forceinline__ float weight_of(float l, bool on, bool sigmoid, bool renormalize,
                                           RowScale r) {
  if (!renormalize) {
    if (!on) return 0.f;
    return sigmoid ? __fdiv_rn(1.f, 1.f + expf(-l)) : __fdiv_rn(expf(l - r.top), r.sum);
  }
  const float top = warp_max(on ? l : -INFINITY);
  if (!sigmoid && r.sum != r.sum) return on ? r.sum : 0.f;  // a NaN among the row's scores
  // sigmoid(l) is exp(l) to the last bit where no logit is above -60, and exp(l - top) does not
  // underflow
  const float p = !on                        ? 0.f
                  : sigmoid && !(top < -60.f) ? __fdiv_rn(1.f, 1.f + expf(-l))
                                              : expf(l - top);
  const float sum = warp_sum(p);
  return on ? __fdiv_rn(p, sum) : 0.f;
}

// A warp a token: lane i holds the logits of V consecutive experts from i V on.
template <typename T, int V>
__global__ void __launch_bounds__(256) route_kernel(const RouteArgs P) {
  extern __shared__ double route_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (token >= P.tokens) return;
  const T* logits = static_cast<const T*>(P.logits) + token * P.stride;
  double* room = route_smem + static_cast<int64_t>(warp) * P.experts;
  const int e0 = lane * V;
  float l[V];
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = e0 + v < P.experts ? to_f32(logits[e0 + v]) : -INFINITY;

  RowScale scale = {0.f, 1.f};
  if (!P.sigmoid && !(P.by_logits && P.renormalize)) {
    float top = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, l[v]);
    scale.top = warp_max(top);
    float part[V];
#pragma unroll
    for (int v = 0; v < V; ++v) part[v] = __expf(l[v] - scale.top);
#pragma unroll
    for (int o = V / 2; o; o >>= 1)
#pragma unroll
      for (int v = 0; v < o; ++v) part[v] += part[v + o];
    scale.sum = warp_sum(part[0]);
  }

  const auto choice_of = [&](float v, int e) {
    if (P.by_logits) return v;
    const float s = score_of(v, P.sigmoid, scale);
    return P.bias ? s + P.bias[e] : s;
  };
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = 0;
    if (e0 + v < P.experts && l[v] != -INFINITY) {
      const float c = choice_of(l[v], e0 + v);
      if (c != -INFINITY) key[v] = order_of(c);
    }
  }

  // Two choices closer than this may be the other way round in exact arithmetic.  A
  // score is off by at most 35 units of 2^-24 of the row's largest possible score
  // (softmax: the exponentials of logit and sum, 4 + 2 |x| units each at x below the top,
  // where exp(x) |x| <= 0.37 and the mean of |x| over the row is at most log 1024, and
  // the sum's ten additions; sigmoid: 6), a sum with the bias by half a unit of its own.
  const float step = (P.sigmoid ? 1.f : __fdividef(1.f, scale.sum)) * 0x1p-17f;
  bool unsure = false;

  if (P.groups > 1) {
    const int size = P.experts / P.groups;
    float* c = reinterpret_cast<float*>(room);
    uint32_t* o = reinterpret_cast<uint32_t*>(room) + P.experts;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v < P.experts) {
        c[e0 + v] = key[v] ? choice_of(l[v], e0 + v) : -INFINITY;
        o[e0 + v] = key[v];
      }
    __syncwarp();
    float worth = -INFINITY;
    uint32_t rank = 0;
    if (lane < P.groups) {
      uint32_t first = 0, second = 0;
      float a = 0.f, b = 0.f;
      for (int i = 0; i < size; ++i) {
        const uint32_t k = o[lane * size + i];
        if (k > first) second = first, b = a, first = k, a = c[lane * size + i];
        else if (k > second) second = k, b = c[lane * size + i];
      }
      if (first) {
        worth = P.group_best > 1 && second ? a + b : a;
        rank = order_of(worth);
      }
    }
    const unsigned open = best_groups(rank, P.groups, P.top_groups);
    if (!P.by_logits && __popc(open) < P.groups) {
      // the least worth that is taken and the largest that is left
      const bool in = open >> lane & 1;
      const bool left = lane < P.groups && !in && rank;
      const float last = -warp_max(in ? -worth : -INFINITY), next = warp_max(left ? worth : -INFINITY);
      const bool odd = __any_sync(kAll, (in || left) && !(fabsf(worth) < INFINITY));
      unsure = __any_sync(kAll, left) &&
               (odd || !(last - next > 2.f * step + 0x1p-21f * fmaxf(fabsf(last), fabsf(next))));
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v < P.experts && !(open >> ((e0 + v) / size) & 1)) key[v] = 0;
    __syncwarp();
  }

  int mine = -1;  // lane j: the j-th expert
  const int rounds = P.by_logits ? P.k : P.k + 1;
  for (int r = 0; r < rounds && !unsure; ++r) {
    uint32_t most = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) most = max(most, key[v]);
    const uint32_t best = __reduce_max_sync(kAll, most);
    if (!best) break;
    const int winner = __ffs(__ballot_sync(kAll, most == best)) - 1;
    int at = 0;
    if (lane == winner) {
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (key[v] == best) at = v;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v == at) key[v] = 0;
    }
    at = __shfl_sync(kAll, at, winner);
    if (lane == r) mine = winner * V + at;
  }
  float chosen = mine >= 0 ? to_f32(logits[mine]) : 0.f;
  if (!P.by_logits && !unsure) {
    // neighbours in the order that fp32 does not tell apart; the same logit and bias tie
    // in any arithmetic
    const float b = P.bias && mine >= 0 ? P.bias[mine] : 0.f;
    const float c = mine >= 0 ? choice_of(chosen, mine) : 0.f;
    const float lp = __shfl_up_sync(kAll, chosen, 1), bp = __shfl_up_sync(kAll, b, 1);
    const float cp = __shfl_up_sync(kAll, c, 1);
    const bool near = lane > 0 && mine >= 0 &&
                      !(cp - c > step + 0x1p-22f * fmaxf(fabsf(c), fabsf(cp))) &&
                      !(lp == chosen && bp == b);
    unsure = __any_sync(kAll, near);
  }
  if (unsure) {
    mine = choose_exactly(P, logits, room);
    chosen = mine >= 0 ? to_f32(logits[mine]) : 0.f;
  }
  if (lane >= P.k) mine = -1;  // the one past the last
  const float w = weight_of(chosen, mine >= 0, P.sigmoid, P.renormalize, scale);
  if (lane < P.k) {
    const int64_t at = token * P.k + lane;
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

// A warp a token: lane j forms the gradient of the j-th expert's logit, the row is
// put together in shared memory and stored.
template <typename T>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteGradArgs P) {
  extern __shared__ float grad_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (token >= P.tokens) return;
  const T* logits = static_cast<const T*>(P.logits) + token * P.stride;
  T* grad = static_cast<T*>(P.grad) + token * P.grad_stride;
  float* row = grad_smem + warp * P.experts;
  for (int e = lane; e < P.experts; e += 32) row[e] = 0.f;
  int64_t id = -1;
  if (lane < P.k) {
    const int64_t at = token * P.k + lane;
    id = P.wide_ids ? static_cast<const int64_t*>(P.ids)[at] : static_cast<const int*>(P.ids)[at];
  }
  const bool on = id >= 0 && id < P.experts;
  const int e = on ? static_cast<int>(id) : -1 - lane;  // no two lanes' alike
  const float l = on ? to_f32(logits[e]) : 0.f;
  const float g = on ? P.scale * P.grad_weights[token * P.k + lane] : 0.f;
  RowScale scale = {0.f, 1.f};
  const bool whole = !P.sigmoid && !P.renormalize;  // every logit has a gradient
  if (whole) {
    float top = -INFINITY;
    for (int i = lane; i < P.experts; i += 32) top = fmaxf(top, to_f32(logits[i]));
    scale.top = warp_max(top);
    float sum = 0.f;
    for (int i = lane; i < P.experts; i += 32) sum += expf(to_f32(logits[i]) - scale.top);
    scale.sum = warp_sum(sum);
  }
  const float p = weight_of(l, on, P.sigmoid, P.renormalize, scale);
  const float mean = P.sigmoid && !P.renormalize ? 0.f : warp_sum(g * p);
  float d = g;
  if (!whole) {
    d = p * (g - mean);
    if (P.sigmoid) d *= __fdiv_rn(1.f, 1.f + expf(l));  // 1 - sigmoid(l)
  }
  __syncwarp();
  const unsigned same = __match_any_sync(kAll, e);
  if (__any_sync(kAll, on && __popc(same) > 1)) {
    for (int j = 0; j < P.k; ++j) {  // an expert named twice: in the order of j
      if (lane == j && on) row[e] += d;
      __syncwarp();
    }
  } else if (on) {
    row[e] = d;
  }
  __syncwarp();
  const auto value = [&](int i) {
    if (!whole) return row[i];
    if (scale.top == -INFINITY) return 0.f;  // every expert is closed
    return __fdiv_rn(expf(to_f32(logits[i]) - scale.top), scale.sum) * (row[i] - mean);
  };
  if (P.vectors) {
    for (int i = lane * kVec<T>; i < P.experts; i += 32 * kVec<T>) {
      float f[kVec<T>];
#pragma unroll
      for (int u = 0; u < kVec<T>; ++u) f[u] = value(i + u);
      store_vec(grad + i, from_floats<T>(f));
    }
  } else {
    for (int i = lane; i < P.experts; i += 32) grad[i] = from_f32<T>(value(i));
  }
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

template <typename T>
tbe_status launch_route(const RouteArgs& args, cudaStream_t s) {
  // choices in 64 bits, or as fp32 and its order
  const size_t row = args.by_logits && args.groups == 1 ? 0 : args.experts * sizeof(double);
  const int warps = args.experts > 512 ? 4 : 8;
  const unsigned ctas = static_cast<unsigned>((args.tokens + warps - 1) / warps);
  const auto go = [&](auto v) {
    route_kernel<T, decltype(v)::value><<<ctas, warps * 32, warps * row, s>>>(args);
    return launched();
  };
  if (args.experts <= 32) return go(std::integral_constant<int, 1>{});
  if (args.experts <= 64) return go(std::integral_constant<int, 2>{});
  if (args.experts <= 128) return go(std::integral_constant<int, 4>{});
  if (args.experts <= 256) return go(std::integral_constant<int, 8>{});
  if (args.experts <= 512) return go(std::integral_constant<int, 16>{});
  return go(std::integral_constant<int, 32>{});
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
                          !bias && (groups == 1 || group_best == 1)};
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
    constexpr int kWarps = 8;
    route_backward_kernel<decltype(t)>
        <<<static_cast<unsigned>((tokens + kWarps - 1) / kWarps), kWarps * 32,
           kWarps * experts * sizeof(float), static_cast<cudaStream_t>(stream)>>>(args);
    return launched();
  });
}
