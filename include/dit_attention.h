/*
 * dit_attention.h -- C ABI of attention, forward and backward, for AMD
 * Instinct MI355X (gfx950): the step between the QK-norm + RoPE pass of
 * qknorm_rope.h and a block's output projection.  The functions are in
 * libdit_attention.so, which libqknorm_rope.so loads (a program that calls them
 * links both).
 *
 * For sample b, query i, head h (which reads key/value head
 * h / (heads / kv_heads)) and the keys j that query i sees:
 *
 *   s_ij  = scale * sum_d q[i, d] k[j, d]
 *   lse_i = log sum_j exp(s_ij)                  p_ij = exp(s_ij - lse_i)
 *   out_i = sum_j p_ij v_j
 *
 * and backwards, with the probabilities computed again from lse:
 *
 *   delta_i = sum_d dout[i, d] out[i, d]
 *   ds_ij   = p_ij (sum_d dout[i, d] v[j, d] - delta_i)
 *   dq_i = scale sum_j ds_ij k_j      dk_j = scale sum_i ds_ij q_i
 *   dv_j = sum_i p_ij dout_i          (dk, dv: summed over the heads that share j's head)
 *
 * Query i sees key j when j < kv_lengths[b] (all keys without kv_lengths) and,
 * if causal, j <= i + kv_tokens - q_tokens (the last query sees the last key).
 * A query that sees no key gets out = 0 and lse = -inf, and adds nothing to
 * any gradient; a key that no query sees gets zero gradients.
 *
 * The products take 16-bit operands and accumulate in fp32: p and ds are
 * rounded to the tensors' type before the products that use them (for up to 32
 * query rows a key head what that leaves is added as a second operand);
 * scores, sums, lse and delta are fp32; each output is rounded once.  For
 * fp16, p and ds are scaled by powers of two into its range first, so neither
 * long rows nor small gradients sink into its subnormals (ds by a bound on its
 * query for dq, by the largest of the key head's queries for dk).  Results do
 * not depend on the order in which workgroups run (no atomic additions).
 *
 * Keys and values at or past kv_lengths[b] are not read.  A query and a key
 * that causality hides from each other may take part in the products with
 * probability 0, so an infinity or NaN in one can reach the other where the key
 * lies less than 192 positions behind the last one that the query sees.
 *
 * All pointers are DEVICE pointers owned by the caller.  The library
 * allocates, frees and synchronises nothing and keeps no state between calls.
 * Work is only enqueued on `stream`.
 */
#ifndef DIT_ATTENTION_H
#define DIT_ATTENTION_H

#include <stdint.h>

#include "qknorm_rope.h" /* status codes and dtype constants */

#ifdef __cplusplus
extern "C" {
#endif

/* One [batch, tokens, heads, head_dim] tensor: element (b, t, h, d) is at
 * data + b * batch_stride + t * token_stride + h * head_stride + d (strides in
 * elements).  The slices of a fused [batch, tokens, 3 * heads * head_dim]
 * buffer are such tensors.  data must be 16-byte aligned, the strides
 * multiples of 8 and not negative, token_stride at least head_dim and at most
 * DIT_ATTN_MAX_TOKEN_STRIDE; the stride of a dimension of one element may be
 * anything.  Elements of an output must not share memory; a batch or head stride
 * of an input may be 0.  A tensor of 0 tokens is not looked at and may be NULL. */
typedef struct {
    void* data;
    int64_t batch_stride, token_stride, head_stride;
} dit_attn_tensor;

#define DIT_ATTN_MAX_TOKEN_STRIDE ((int64_t)1 << 22)

/* What a call computes.  heads * (q_tokens / 32 + 1) and kv_heads *
 * (kv_tokens / 32 + 1), times batch, must stay below 2^23, and q_tokens * heads
 * / kv_heads below 2^30. */
typedef struct {
    int64_t batch;              /* 0 is a no-op                                       */
    int64_t q_tokens;           /* 0 .. QKR_MAX_TOKENS - 1                            */
    int64_t kv_tokens;          /* 0 .. QKR_MAX_TOKENS - 1                            */
    int32_t heads;              /* query heads, a multiple of kv_heads                */
    int32_t kv_heads;           /* 1 .. QKR_MAX_HEADS                                 */
    int32_t head_dim;           /* 64, 128 or 256                                     */
    int32_t causal;             /* 0 or 1                                             */
    int32_t dtype;              /* QKR_BF16 or QKR_FP16, of every tensor but lse      */
    float scale;                /* > 0, finite also times log2(e)                     */
    const int32_t* kv_lengths;  /* device array [batch], or NULL; a length below 0    */
                                /* counts as 0, one above kv_tokens as kv_tokens      */
} dit_attn_args;

/* Bytes of workspace the calls need for these sizes (0: none), or a negative
 * QKR_ERR_* code.  The workspace is scratch: 16-byte aligned, its contents are
 * not read before they are written, and it must not be shared by calls that
 * may run at the same time. */
int64_t dit_attention_workspace_size(const dit_attn_args* args);
int64_t dit_attention_backward_workspace_size(const dit_attn_args* args);

/*
 * dit_attention -- out and lse from q, k and v.
 * lse: fp32 [batch, heads, q_tokens], contiguous.
 * Returns QKR_OK or a negative QKR_ERR_* code; all checks happen before any
 * HIP call and nothing is enqueued on error.  QKR_ERR_ARG also when an output
 * may overlap another tensor of the call or itself.
 */
int dit_attention(const dit_attn_args* args, const dit_attn_tensor* q, const dit_attn_tensor* k,
                  const dit_attn_tensor* v, const dit_attn_tensor* out, float* lse,
                  void* workspace, int64_t workspace_bytes, void* stream);

/*
 * dit_attention_backward -- dq, dk and dv (written, not added to) from dout
 * and the forward call's tensors.  Every element of dq, dk and dv is written,
 * zeros where the masks leave nothing.
 */
int dit_attention_backward(const dit_attn_args* args, const dit_attn_tensor* dout,
                           const dit_attn_tensor* q, const dit_attn_tensor* k,
                           const dit_attn_tensor* v, const dit_attn_tensor* out, const float* lse,
                           const dit_attn_tensor* dq, const dit_attn_tensor* dk,
                           const dit_attn_tensor* dv, void* workspace, int64_t workspace_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DIT_ATTENTION_H */
