/*
 * qknorm_rope_backward.h -- C ABI of the backward pass of the fused QK-norm +
 * RoPE pass of qknorm_rope.h, built into the same library.
 *
 * With x the pass's input (before it was written over), o its output, do the
 * gradient of o, r = 1 / sqrt(mean_d x[d]^2 + eps) and u = x r:
 *
 *   dn[a] = do[a] cos[a] + do[b] sin[b]       the transposed rotation, for each
 *   dn[b] = do[b] cos[b] - do[a] sin[a]       rotary pair (a, b)
 *   g = dn * gamma
 *   dx[d] = r (g[d] - u[d] mean_e(g[e] u[e]))
 *   dgamma[d] = sum over tokens and heads of dn[d] u[d]
 *
 * separately for Q and K.  cos and sin are tables and get no gradient.  Math
 * is fp32; dx is rounded once, to nearest even; dgamma is an fp32 sum in an
 * order that depends on the sizes alone.  Any finite x is handled, as
 * qknorm_rope.h describes, as long as the sums of |g| over a head stay in
 * fp32's range.
 *
 * Pointers are DEVICE pointers owned by the caller; the library allocates,
 * frees and synchronises nothing and work is only enqueued on `stream`.
 */
#ifndef QKNORM_ROPE_BACKWARD_H
#define QKNORM_ROPE_BACKWARD_H

#include <stdint.h>

#include "qknorm_rope.h" /* status codes, dtype, layout and style constants */

#ifdef __cplusplus
extern "C" {
#endif

/* Workgroups over which a call spreads its tokens, at most, each with a row of
 * the workspace for its sums of dgamma. */
#define QKR_BACKWARD_MAX_BLOCKS 2048

/* The gradient, input and output tensors of one of the forms of a call. */
typedef struct {
    const void* grad;   /* do                                                       */
    const void* x;      /* the forward pass's input                                 */
    void* out;          /* dx; may be grad itself (in place), overlaps nothing else */
} qkr_grad_tensor;

/* Bytes of workspace a call for `tokens` tokens of head_dim needs, or a
 * negative QKR_ERR_* code. */
int64_t qknorm_rope_backward_workspace_size(int64_t tokens, int32_t head_dim);

/*
 * qknorm_rope_backward
 *
 * Modes (exactly one), each tensor laid out as in qknorm_rope_fused:
 *   fused:    qkv != NULL, q == k == NULL: grad, x and out are [tokens,
 *             3*heads*head_dim] buffers whose Q and K slices are read and
 *             written; the V slices are neither.
 *   separate: qkv == NULL and at least one of q, k != NULL, of [tokens, heads,
 *             head_dim] tensors; a tensor that is NULL is skipped, and its gamma
 *             and dgamma may be NULL.
 * q_gamma, k_gamma      fp32 [head_dim].
 * dq_gamma, dk_gamma    fp32 [head_dim], written (not added to).
 * tokens                0 writes zeros to dq_gamma and dk_gamma.
 * workspace             16-byte aligned scratch of at least the queried size, not
 *                       shared by calls that may run at the same time.
 * The other arguments are qknorm_rope_fused's.  Every pointer must be 16-byte
 * aligned.  Returns QKR_OK or a negative QKR_ERR_* code; all checks happen
 * before any HIP call and nothing is enqueued on error.
 */
int qknorm_rope_backward(const qkr_grad_tensor* qkv, const qkr_grad_tensor* q,
                         const qkr_grad_tensor* k, int64_t tokens, int32_t heads, int32_t head_dim,
                         const float* q_gamma, const float* k_gamma, float* dq_gamma,
                         float* dk_gamma, float eps, const void* cos, const void* sin,
                         int32_t cos_layout, int32_t cos_dtype, int32_t style, int32_t dtype,
                         void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QKNORM_ROPE_BACKWARD_H */
