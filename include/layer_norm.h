/*
 * layer_norm.h -- C ABI of layer norm, forward and backward, for AMD Instinct
 * MI355X (gfx950), built into the same library as qknorm_rope.h.  The backward
 * pass also serves the modulated form of fuse_scale_shift.h.
 *
 *   for row r of x [rows, hidden]:
 *     mean, var    of the row (biased variance)
 *     n[c] = (x[c] - mean) / sqrt(var + eps)
 *     y[c] = n[c] * weight[c] + bias[c]
 *
 * and backwards, with w the weight row that r uses and g = dy * w:
 *     dx[c] = (g[c] - avg(g) - n[c] avg(g n)) / sqrt(var + eps)
 *     dweight[c] = sum_r dy[c] n[c]          dbias[c] = sum_r dy[c]
 *
 * The backward pass computes mean and var again from x, which it reads anyway,
 * so the forward pass leaves nothing behind for it.
 *
 * Math is fp32; y and dx are rounded once, to nearest even, to x's dtype;
 * dweight and dbias are fp32 sums in an order that depends on the sizes alone,
 * so results do not change from run to run.  Rows of any finite values are
 * normalised correctly, as fuse_scale_shift.h describes, and get their
 * gradients, as long as the sums of |g| over a row stay in fp32's range (bf16
 * gradients of 1e34 may leave it; the row's dx is then infinite or NaN).
 *
 * Pointers are DEVICE pointers owned by the caller; the library allocates,
 * frees and synchronises nothing and work is only enqueued on `stream`.
 */
#ifndef LAYER_NORM_H
#define LAYER_NORM_H

#include <stdint.h>

#include "qknorm_rope.h" /* status codes and dtype constants */

#ifdef __cplusplus
extern "C" {
#endif

#define DIT_LN_MAX_HIDDEN 8192   /* hidden must be a multiple of 8 in [8, 8192] */

/* What the backward pass's weight tensor holds. */
enum {
    DIT_LN_WEIGHT = 0,     /* w itself (dit_layer_norm)                          */
    DIT_LN_ONE_PLUS = 1    /* w - 1: the scale of dit_fuse_scale_shift           */
};

/*
 * dit_layer_norm
 *
 * x, y          [rows, hidden] contiguous, dtype QKR_BF16 or QKR_FP16; y may be
 *               x itself or a buffer that does not overlap it.
 * rows          >= 0 (0 is a no-op once scalars are valid), below QKR_MAX_TOKENS.
 * hidden        multiple of 8, 8 .. DIT_LN_MAX_HIDDEN.
 * weight, bias  [hidden] of param_dtype (QKR_BF16, QKR_FP16 or QKR_FP32); either
 *               may be NULL (all ones, all zeros).
 * eps           finite and > 0.
 *
 * Every pointer must be 16-byte aligned.  Returns QKR_OK or a negative
 * QKR_ERR_* code; all checks happen before any HIP call.
 */
int dit_layer_norm(const void* x, void* y, int64_t rows, int32_t hidden, const void* weight,
                   const void* bias, int32_t param_dtype, float eps, int32_t dtype, void* stream);

/* Bytes of workspace that dit_layer_norm_backward needs when it computes
 * dweight and dbias (0: none), or a negative QKR_ERR_* code. */
int64_t dit_layer_norm_backward_workspace_size(int64_t rows, int32_t hidden,
                                               int64_t rows_per_batch);

/*
 * dit_layer_norm_backward
 *
 * dy, x, dx       [rows, hidden] contiguous; dx may be dy itself, and overlaps
 *                 nothing else.
 * rows_per_batch  >= 1; row r uses weight row r / rows_per_batch, and its sums
 *                 go to that row of dweight and dbias (one row for all: any
 *                 value >= rows).
 * weight          [ceil(rows / rows_per_batch), hidden] of param_dtype, or NULL
 *                 (all ones); weight_form says what it holds.
 * dweight, dbias  fp32 [ceil(rows / rows_per_batch), hidden], written (not added
 *                 to); both or neither.  They overlap no other buffer.
 * workspace       16-byte aligned scratch of at least the queried size when
 *                 dweight is given, not shared by calls that may run at the same
 *                 time.
 * With rows == 0 nothing is written.
 */
int dit_layer_norm_backward(const void* dy, const void* x, void* dx, int64_t rows, int32_t hidden,
                            int64_t rows_per_batch, const void* weight, int32_t weight_form,
                            int32_t param_dtype, float* dweight, float* dbias, float eps,
                            int32_t dtype, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYER_NORM_H */
