/*
 * tbe_norm.h -- C ABI of the root-mean-square norm of the GB300 (sm_103a)
 * Table Batched Embedding library: the norm with the residual's addition, its
 * output in the rows' type or in 8 bits with scales, and its gradients.
 *
 *   h[r] = rn(x[r] + residual[r])                 x[r] itself without a residual
 *   u[r] = 1 / sqrt(sum_c h[r, c]^2 / H + eps)
 *   y[r, c] = rn(h[r, c] * u[r] * weight[c])
 *
 * R rows of H columns, 1 <= H <= TBE_MAX_NORM_WIDTH.  The norm is of the sum as
 * it is held in the rows' type, so that the gradients, which read h, belong to it.
 * Squares, sums and products are fp32 (a square above 2^128 overflows: u = 0; one below
 * 2^-149 is lost, which shows where eps is no larger); each result is rounded once.  A row
 * of zeros with eps = 0 follows the formula (NaN).
 *
 * Matrices are row-major with a row stride in elements (at least the row's columns);
 * their columns are contiguous.  dtype (x, residual, h, y and the gradients of rows) is
 * TBE_DT_F16, TBE_DT_BF16 or TBE_DT_F32; weight is contiguous [H] of weight_dtype, which is
 * dtype or TBE_DT_F32; NULL: ones.  No output may share memory with an input or another
 * output.
 *
 * Ordering, allocation and errors follow tbe.h: every call only enqueues work on
 * the given stream, allocates nothing, can be captured into a CUDA graph, and
 * reports argument problems before anything is enqueued.  No atomics: the same call
 * gives the same bits (sums are in an order that the sizes and the alignment of the
 * rows set).
 * Errors: TBE_EINVAL (null pointers, sizes, strides, alignment, shared memory, an eps that
 * is negative or not finite), TBE_EUNSUPPORTED (types, H > TBE_MAX_NORM_WIDTH, R >= 2^31),
 * TBE_EWORKSPACE, TBE_ECUDA.
 */
#ifndef TBE_NORM_H_
#define TBE_NORM_H_

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TBE_MAX_NORM_WIDTH 16384

/* The norm in the rows' own type: y [R, H].  residual NULL: none.  h [R, H] or NULL:
 * where the sum goes. */
tbe_status tbe_rms_norm(const void* x, const void* residual, const void* weight, int32_t dtype,
                        int32_t weight_dtype, int64_t rows, int64_t width, int64_t x_stride,
                        int64_t residual_stride, float eps, void* h, int64_t h_stride, void* y,
                        int64_t y_stride, void* stream);

/* The norm quantised to e4m3 with one scale for each 128 columns of a row, as
 * tbe_expert_product takes it (the arithmetic of tbe_quantize_weights in
 * tbe_experts.h, on the unrounded fp32 products h * u * weight):
 * q [R, H] one byte a value, scale [R, ceil(H / 128)] fp32 (contiguous).
 * It is for products of all rows with one expert.  Experts that a router chooses take
 * rows sorted by expert, which no call here makes of 8-bit rows, and the router itself needs y:
 * there take tbe_rms_norm, and tbe_expert_dispatch_fp8 quantises the rows on their way. */
tbe_status tbe_rms_norm_fp8(const void* x, const void* residual, const void* weight,
                            int32_t dtype, int32_t weight_dtype, int64_t rows, int64_t width,
                            int64_t x_stride, int64_t residual_stride, float eps, void* h,
                            int64_t h_stride, uint8_t* q, int64_t q_stride, float* scale,
                            void* stream);

/* Scratch of tbe_rms_norm_backward with grad_weight: device memory, 16-byte aligned,
 * any contents. */
tbe_status tbe_rms_norm_workspace_size(int64_t rows, int64_t width, size_t* bytes);

/* Gradients of tbe_rms_norm (and of tbe_rms_norm_fp8 taken as the norm):
 *   d[r, c] = grad_y[r, c] * weight[c]
 *   grad_x[r, c] = rn(u[r] * (d[r, c] - h[r, c] * u[r] * sum_i d[r, i] h[r, i] u[r] / H)
 *                     + grad_h[r, c])
 *   grad_weight[c] = sum_r grad_y[r, c] * h[r, c] * u[r]
 * grad_x is the gradient of x and of residual alike.  grad_h: the gradient that
 * arrives at h, NULL: none.  grad_weight fp32 [H], summed in fp32, or NULL (workspace is
 * then not used).  h: tbe_rms_norm's, or x where it had no residual.  rows = 0 gives
 * grad_weight zeros. */
tbe_status tbe_rms_norm_backward(const void* grad_y, const void* h, const void* weight,
                                 const void* grad_h, int32_t dtype, int32_t weight_dtype,
                                 int64_t rows, int64_t width, int64_t grad_y_stride,
                                 int64_t h_stride, int64_t grad_h_stride, float eps, void* grad_x,
                                 int64_t grad_x_stride, float* grad_weight, void* workspace,
                                 size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_NORM_H_ */
