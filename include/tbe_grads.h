/*
 * tbe_grads.h -- C ABI of the gradient-norm operators of the GB300 (sm_103a)
 * Table Batched Embedding library: the global norm over many gradients, and
 * the gradients clipped to a largest norm.
 *
 *   norm  = sqrt(sum over tensors t, elements i of g_t[i]^2)
 *   c     = min(1, max_norm / (norm + 1e-6))
 *   out_t = rn(c * g_t)
 *
 * The norm holds over the whole range of fp32: each thread's short fp32 sums
 * of squares are formed again with a power-of-two factor where they leave
 * [2^-60, 2^100], and are joined in fp64 in an order that depends on the sizes
 * and on where in 16 bytes each tensor begins: the same call gives the same
 * bits.  An infinity or NaN among the gradients makes the norm infinite or
 * NaN, and c then follows the formula (0, or NaN).
 *
 * Ordering, allocation and errors follow tbe.h.
 */
#ifndef TBE_GRADS_H_
#define TBE_GRADS_H_

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One gradient: numel contiguous elements of dtype (TBE_DT_F16, TBE_DT_BF16 or
 * TBE_DT_F32, aligned to its element).  out: where its clipped values go, of
 * the same type; grad itself for in place.  Otherwise no out may overlap a
 * gradient or another out. */
typedef struct tbe_grad_tensor {
  const void* grad;
  void* out;       /* not used by tbe_grad_norm */
  int64_t numel;
  int32_t dtype;
  int32_t reserved;
} tbe_grad_tensor;

/* Scratch both calls need: device memory, 16-byte aligned, any contents. */
#define TBE_GRAD_WORKSPACE_BYTES 16384u

/* tensors: a host array, read before the call returns (the addresses travel
 * with the launches).  norm: fp32, device.  count = 0 gives norm 0.
 * Errors: TBE_EINVAL (null pointers, negative sizes, misaligned addresses),
 * TBE_EWORKSPACE, TBE_EUNSUPPORTED (type, or numel > 2^40), TBE_ECUDA. */
tbe_status tbe_grad_norm(const tbe_grad_tensor* tensors, int64_t count, float* norm,
                         void* workspace, size_t ws_bytes, void* stream);

/* As tbe_grad_norm, and the clipped gradients.  Where c is 1 a tensor that is
 * clipped in place is left as it is.  max_norm must not be negative or NaN. */
tbe_status tbe_grad_clip(const tbe_grad_tensor* tensors, int64_t count, float max_norm,
                         float* norm, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_GRADS_H_ */
