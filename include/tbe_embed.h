/*
 * tbe_embed.h -- C ABI of the token embedding of the GB300 (sm_103a) Table
 * Batched Embedding library: one row of a table for each token, scaled, and the
 * table's gradient as a result of its own (tbe.h pools bags of rows and applies
 * its gradient to the tables; here a row is looked up in the table's type, and the
 * gradient is returned for any optimizer, or added to one that a tied output
 * layer has left).
 *
 *   out[n] = rn(scale * table[ids[n]])                       zeros where ids[n] is no row
 *   grad_table[v] = rn(scale * sum over n, ids[n] = v, of grad_out[n])
 *
 * N tokens, V rows of H columns.  Matrices are row-major with a row stride in
 * elements (at least the row's columns); their columns are contiguous.  dtype is
 * TBE_DT_F16, TBE_DT_BF16 or TBE_DT_F32; ids are contiguous TBE_DT_I32 or TBE_DT_I64: an id
 * outside [0, V) names no row (padding).  No output may share memory with an input.
 *
 * Ordering, allocation and errors follow tbe.h: every call only enqueues work on
 * the given stream, allocates nothing, can be captured into a CUDA graph, and
 * reports argument problems before anything is enqueued.  No atomics on results:
 * the same inputs give the same bits.
 * Errors: TBE_EINVAL (null pointers, sizes, strides, alignment, shared memory, a scale that
 * is not finite), TBE_EUNSUPPORTED (types; N or V >= 2^31 - 1025, H > 2^20), TBE_EWORKSPACE,
 * TBE_ECUDA.
 */
#ifndef TBE_EMBED_H_
#define TBE_EMBED_H_

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* table [V, H], out [N, H] of the same type. */
tbe_status tbe_embed(const void* table, int32_t dtype, int64_t rows, int64_t width,
                     int64_t table_stride, const void* ids, int32_t index_dtype, int64_t tokens,
                     float scale, void* out, int64_t out_stride, void* stream);

/* Scratch of tbe_embed_backward: device memory, 16-byte aligned, any contents; none (bytes 0)
 * up to 1024 tokens. */
tbe_status tbe_embed_workspace_size(int64_t tokens, int64_t rows, int64_t width, size_t* bytes);

/* grad_out [N, H] of dtype, grad_table [V, H] of out_dtype, which is dtype or TBE_DT_F32.
 * The tokens are sorted by row; a row's tokens are summed in fp32, in their order
 * within pieces that the sizes set, and rounded once.  accumulate = 0: rows without tokens
 * are zeros.  Otherwise grad_table[v] = rn(grad_table[v] + scale * sum), and rows without
 * tokens are left as they are. */
tbe_status tbe_embed_backward(const void* grad_out, int32_t dtype, int64_t tokens, int64_t width,
                              int64_t grad_out_stride, const void* ids, int32_t index_dtype,
                              int64_t rows, float scale, int32_t accumulate, void* grad_table,
                              int32_t out_dtype, int64_t grad_table_stride, void* workspace,
                              size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_EMBED_H_ */
