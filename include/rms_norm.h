/*
 * rms_norm.h -- C ABI of RMS norm over whole rows, with the residual's addition
 * and an output in 8 bits, and of its backward pass, for AMD Instinct MI355X
 * (gfx950), built into the same library as qknorm_rope.h.
 *
 *   for row r of x [rows, hidden]:
 *     s[c] = x[c] + residual[c], rounded to x's type     (s = x without a residual)
 *     y[c] = s[c] / sqrt(avg(s^2) + eps) * weight[c]
 *
 * or in 8 bits (e4m3, the OCP format: 448 is its largest number), with one
 * scale a row, so that y[c] is y8[c] * scale:
 *     t[c]  = s[c] * weight[c]                 top = max |t|
 *     y8[c] = round(t[c] * (448 / top))        scale = top / sqrt(avg(s^2) + eps) / 448
 * (448 in the place of 448 / top where top is 0).  The values in 8 bits do not
 * depend on the norm, which cancels: it goes into the scale alone.
 *
 * and backwards, with n[c] = s[c] / sqrt(avg(s^2) + eps) and g = dy * weight:
 *     dx[c] = (g[c] - n[c] avg(g n)) / sqrt(avg(s^2) + eps) + dsum[c]
 *     dweight[c] = sum_r dy[c] n[c]
 * dsum is the gradient that reaches s by another way (the residual stream's);
 * dx is the gradient of x and of the residual alike.
 *
 * Math is fp32; s, y and dx are rounded once, to nearest even; dweight is an
 * fp32 sum in an order that depends on the sizes alone, so results do not
 * change from run to run.  Rows of any finite values are normalised correctly
 * (where the plain sums leave fp32's range they are taken again of x * 2^-e, and
 * products t below it of their mantissas) and get their gradients, as long as the products dy * weight stay in fp32's
 * range.  A row that holds a NaN comes out as NaN; with an infinity, finite
 * elements come out as 0 and infinite ones as NaN, and in 8 bits the scale is
 * NaN either way.
 *
 * Pointers are DEVICE pointers owned by the caller; the library allocates,
 * frees and synchronises nothing and work is only enqueued on `stream`.
 */
#ifndef RMS_NORM_H
#define RMS_NORM_H

#include <stdint.h>

#include "qknorm_rope.h" /* status codes and dtype constants */

#ifdef __cplusplus
extern "C" {
#endif

#define DIT_RMS_MAX_HIDDEN 8192   /* hidden must be a multiple of 8 in [8, 8192] */

/*
 * dit_rms_norm
 *
 * x, residual   [rows, hidden] contiguous, dtype QKR_BF16 or QKR_FP16; residual
 *               may be NULL.
 * sum           [rows, hidden], receives s; given if residual is, NULL without.
 *               May be x or residual itself.
 * y             [rows, hidden] of dtype, or, when scales is given, of e4m3 bytes.
 *               Of dtype it may be x or residual itself.
 * scales        fp32 [rows], or NULL for an output of dtype.
 * rows          >= 0 (0 is a no-op once scalars are valid), below QKR_MAX_TOKENS.
 * hidden        multiple of 8, 8 .. DIT_RMS_MAX_HIDDEN.
 * weight        [hidden] of param_dtype (QKR_BF16, QKR_FP16 or QKR_FP32), or NULL
 *               (all ones).
 * eps           finite and > 0.
 *
 * Apart from what is named above no output may overlap another buffer.  Every
 * pointer must be 16-byte aligned (scales: 4).  Returns QKR_OK or a negative
 * QKR_ERR_* code; all checks happen before any HIP call.
 */
int dit_rms_norm(const void* x, const void* residual, void* sum, void* y, float* scales,
                 int64_t rows, int32_t hidden, const void* weight, int32_t param_dtype, float eps,
                 int32_t dtype, void* stream);

/* Bytes of workspace that dit_rms_norm_backward needs when it computes dweight
 * (0: none), or a negative QKR_ERR_* code. */
int64_t dit_rms_norm_backward_workspace_size(int64_t rows, int32_t hidden);

/*
 * dit_rms_norm_backward
 *
 * dy, s, dx   [rows, hidden] contiguous; s is what was normalised (x, or sum).
 * dsum        [rows, hidden], or NULL.  dx may be dy or dsum itself, and overlaps
 *             nothing else.
 * dweight     fp32 [hidden], written (not added to), or NULL; overlaps nothing.
 * workspace   16-byte aligned scratch of at least the queried size when dweight is
 *             given, not shared by calls that may run at the same time.
 * With rows == 0 nothing is written.
 */
int dit_rms_norm_backward(const void* dy, const void* s, const void* dsum, void* dx, int64_t rows,
                          int32_t hidden, const void* weight, int32_t param_dtype, float* dweight,
                          float eps, int32_t dtype, void* workspace, int64_t workspace_bytes,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RMS_NORM_H */
