/*
 * tbe_experts.h -- C ABI of the expert-layer operators of the GB300 (sm_103a)
 * Table Batched Embedding library.
 *
 * A pooled vector (a token) goes to k of E expert networks and comes back as
 * their weighted sum.  The calls below choose the k experts from a router's
 * logits and give the choice's gradient, sort the tokens' assignments by expert,
 * carry the rows there and back, give the gradients of both, quantise rows
 * and weights to 8 bits, and form the experts' matrix products in 8 bits.
 *
 * Notation: N tokens, k assignments per token, A = N k assignments (flat
 * assignment a = n k + j), E experts, H columns.  Every buffer is a device
 * buffer owned by the caller.  Matrices are row-major with a row stride in
 * elements (at least the row's columns); their columns are contiguous.
 * Row data types are TBE_DT_F16, TBE_DT_BF16 and TBE_DT_F32.
 *
 * No output may share memory with an input or with another output of its call.
 * Columns of one buffer may lie beside columns of another.  Shared matrices, ids
 * and positions are refused (TBE_EINVAL); matrices whose row strides differ
 * count as shared where their columns meet modulo the strides' greatest common
 * divisor.
 *
 * Ordering, allocation and errors follow tbe.h: every call only enqueues work
 * on the given stream and returns, allocates nothing, can be captured into a
 * CUDA graph, and reports argument problems through tbe_status before
 * anything is enqueued.  No atomics on results: the same inputs give the same
 * bits.
 */
#ifndef TBE_EXPERTS_H_
#define TBE_EXPERTS_H_

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TBE_MAX_EXPERTS 1024   /* experts of one call */
#define TBE_SCALE_BLOCK 128    /* columns (and weight rows) that share a scale */
#define TBE_MAX_CHOSEN 31      /* experts chosen for one token */

enum { TBE_SCORE_SOFTMAX = 1, TBE_SCORE_SIGMOID = 2 };

/* Chooses k experts for each token and weights them.  logits [N, E] of dtype:
 *   s[n, e] = softmax over e, or sigmoid, of logits[n, e]
 *   c[n, e] = s[n, e] + bias[e]                   bias fp32 [E], or NULL
 * An expert is closed to a token where its logit or c is -inf: its score is then s as it
 * is, and it is not chosen.  With G > 1 groups of E / G consecutive experts, a group is worth
 * the sum of its group_best (1 or 2) largest c (of those that are open), and only the top_groups
 * groups that are worth most are open.  The k open experts with the largest c are
 * chosen, in that order:
 *   ids [N, k]      of index_dtype; -1 where fewer are open (tbe_expert_sort drops those)
 *   weights [N, k]  fp32: scale * s, or with renormalize scale * s / (sum of the chosen s);
 *                   0 where ids is -1
 * Ties go to the lower expert or group.  The choice is that of exact arithmetic
 * wherever 64 bits tell the c apart: where fp32 does not, it is made again in 64 bits.
 * Without a bias the experts' logits themselves are compared.  The bias only chooses: weights
 * are of s, in fp32 by exponentials to two units in the last place and rounded divisions, in
 * tbe_expert_route_backward too.  NaN ranks above everything, so a token with a NaN logit
 * shows it in its weights; softmax of +inf is NaN as the formula gives, and a row that is
 * closed throughout has ids -1.
 * logits have a row stride in elements; ids and weights are contiguous.
 * Errors: TBE_EINVAL (sizes: k > top_groups * E / G, E not a multiple of G, ...; a scale that is
 * not finite), TBE_EUNSUPPORTED (types, E > TBE_MAX_EXPERTS, k > TBE_MAX_CHOSEN, G > 32,
 * N >= 2^31 / k), TBE_ECUDA. */
tbe_status tbe_expert_route(const void* logits, int32_t dtype, int64_t tokens, int32_t experts,
                            int64_t logits_stride, const float* bias, int32_t score, int32_t k,
                            int32_t groups, int32_t top_groups, int32_t group_best,
                            int32_t renormalize, float scale, void* ids, int32_t index_dtype,
                            float* weights, void* stream);

/* Gradient of tbe_expert_route's weights in the logits (the choice has none):
 *   grad_logits[n, e] = rn(sum_j grad_weights[n, j] * d weights[n, j] / d logits[n, e])
 * for the ids [N, k] given; an id outside [0, E) takes no part, and what its
 * grad_weights holds is not used.  An expert may be named twice.  grad_logits [N, E] of
 * dtype. */
tbe_status tbe_expert_route_backward(const float* grad_weights, const void* logits, int32_t dtype,
                                     int64_t tokens, int32_t experts, int64_t logits_stride,
                                     const void* ids, int32_t index_dtype, int32_t k,
                                     int32_t score, int32_t renormalize, float scale,
                                     void* grad_logits, int64_t grad_stride, void* stream);

/* Sorts the assignments by expert, stably (within an expert in the order of
 * a).  ids [N, k] (contiguous, TBE_DT_I32 or TBE_DT_I64): an id outside [0, E)
 * drops its assignment.
 *   offsets [E + 1]   assignments of experts before e; offsets[E] = M kept ones
 *   source [A]        flat assignment of each sorted place r < M; -1 from M on
 *   position [N, k]   sorted place of each assignment; -1 if dropped
 * Errors: TBE_EINVAL, TBE_EUNSUPPORTED (A >= 2^31, E > TBE_MAX_EXPERTS, index
 * type), TBE_ECUDA. */
tbe_status tbe_expert_sort(const void* ids, int32_t index_dtype, int64_t tokens, int32_t k,
                           int32_t experts, int32_t* offsets, int32_t* source, int32_t* position,
                           void* stream);

/* Carries the tokens' rows to their experts:
 *   rows[position[n, j]] = x[n];   rows[r] = 0 for M <= r < A
 * x [N, H], rows [A, H].  offsets and position are tbe_expert_sort's;
 * positions outside [0, A) count as dropped, here and in every call below.
 * Errors: TBE_EINVAL, TBE_EUNSUPPORTED, TBE_ECUDA. */
tbe_status tbe_expert_dispatch(const void* x, int32_t dtype, int64_t tokens, int32_t k,
                               int64_t width, int64_t x_stride, const int32_t* offsets,
                               int32_t experts, const int32_t* position, void* rows,
                               int64_t rows_stride, void* stream);

/* The same with the rows quantised to e4m3 on the way, one scale for each 128
 * columns of a row (the arithmetic of tbe_quantize_weights): q [A, H] one byte
 * a value, scale [A, ceil(H / 128)] fp32 (contiguous).  Rows from M on: q = 0 and
 * scale = 2^-126, what a row of zeros gives.  position may be NULL with k = 1
 * (every row stays where it is; offsets is not read then). */
tbe_status tbe_expert_dispatch_fp8(const void* x, int32_t dtype, int64_t tokens, int32_t k,
                                   int64_t width, int64_t x_stride, const int32_t* offsets,
                                   int32_t experts, const int32_t* position, uint8_t* q,
                                   int64_t q_stride, float* scale, void* stream);

/* Brings the experts' rows back, weighted:
 *   out[n] = rn(sum_j weights[n, j] * y[position[n, j]])
 * over the kept assignments, summed in fp32 in the order of j and rounded
 * once; a token with no kept assignment gets zeros.  What a dropped
 * assignment's weight holds is not used.  y [A, H], weights fp32 [N, k]
 * (contiguous) or NULL for ones, out [N, H].  With weights NULL and y the
 * gradient of tbe_expert_dispatch's rows, out is the gradient of its x. */
tbe_status tbe_expert_combine(const void* y, int32_t dtype, int64_t tokens, int32_t k,
                              int64_t width, int64_t y_stride, const int32_t* position,
                              const float* weights, void* out, int64_t out_stride, void* stream);

/* Gradients of tbe_expert_combine:
 *   grad_y[position[n, j]] = rn(weights[n, j] * grad_out[n]);  0 for rows M..A-1
 *   grad_weights[n, j] = sum_h grad_out[n, h] * y[position[n, j], h]   (fp32; 0 if dropped)
 * weights NULL: ones.  grad_y may be NULL, and so may grad_weights (y is then
 * not read and may be NULL). */
tbe_status tbe_expert_combine_backward(const void* grad_out, const void* y, int32_t dtype,
                                       int64_t tokens, int32_t k, int64_t width,
                                       int64_t grad_out_stride, int64_t y_stride,
                                       const int32_t* offsets, int32_t experts,
                                       const int32_t* position, const float* weights,
                                       void* grad_y, int64_t grad_y_stride, float* grad_weights,
                                       void* stream);

/* Quantises weights [E, N, K] (contiguous) to e4m3 with one scale for each
 * 128 x 128 block of an expert's matrix:
 *   scale = max(amax * (1/448), 2^-126);  q = e4m3(w / scale)
 * in fp32, with 1/448 rounded to fp32, the division rounded to nearest and the
 * values rounded to nearest even (448 is the largest).
 * q [E, N, K]; scale fp32 [E, ceil(N / 128), ceil(K / 128)].  An infinity
 * gives its block an infinite scale; a NaN stays one NaN value.
 * Errors: TBE_EINVAL, TBE_EUNSUPPORTED (type; N or K above 2^31 - 513, or 2^31
 * blocks), TBE_ECUDA. */
tbe_status tbe_quantize_weights(const void* w, int32_t dtype, int64_t experts, int64_t n,
                                int64_t k, uint8_t* q, float* scale, void* stream);

/* The experts' products on 8-bit rows and weights:
 *   out[r, n] = rn(sum_b a_scale[r, b] * w_scale[e, n / 128, b]
 *                        * sum_{i in block b} a[r, i] * w[e, n, i])
 * for offsets[e] <= r < offsets[e + 1], and out[r] = 0 for the other rows, those
 * before offsets[0] and from offsets[E] on.  The inner sums and the sum over
 * blocks are fp32; the two scales are multiplied first, in fp32, so a product of
 * scales below 2^-126 loses bits.
 * a [rows, K] e4m3 with a_scale [rows, ceil(K / 128)] (contiguous); w
 * [E, N, K] e4m3 (contiguous) with w_scale [E, ceil(N / 128), ceil(K / 128)]
 * (contiguous); offsets [E + 1], or NULL with E = 1 for all rows; out
 * [rows, N] of out_dtype.  The gradient of the rows is the same product with
 * the transposed weights [E, K, N] (quantised in the same blocks, so they
 * hold the same values).  K, a_stride and the addresses of a and w must be
 * multiples of 16 (16-byte copies).
 * offsets are clamped into [0, rows], whatever they hold; an expert whose end
 * lies before its start has no rows.  Where offsets do not rise, what out holds
 * is not defined (nothing outside it is written).
 * status: device int32 word, or NULL.  A bounded device wait that gave up sets
 * TBE_ERR_TIMEOUT in it, and with or without it every element of out that may
 * be lost is NaN.
 * Errors: TBE_EINVAL, TBE_EUNSUPPORTED (type; alignment; rows, K or E N above
 * 2^31 - 513, E > TBE_MAX_EXPERTS, or too many tiles), TBE_ECUDA. */
tbe_status tbe_expert_product(const uint8_t* a, int64_t a_stride, const float* a_scale,
                              const uint8_t* w, const float* w_scale, const int32_t* offsets,
                              int64_t rows, int64_t n, int64_t k, int32_t experts, void* out,
                              int32_t out_dtype, int64_t out_stride, int32_t* status,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_EXPERTS_H_ */
