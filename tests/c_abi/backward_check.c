/* Plain C consumer of the headers of attention, layer norm and the backward
 * passes: compiled with gcc by tests/test_backward_c_abi.py and run on the CPU.
 * Every call is rejected before any HIP call or has nothing to do.  Prints
 * "ok" and exits 0 when every code matches. */
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "dit_attention.h"
#include "layer_norm.h"
#include "qknorm_rope_backward.h"

#define EXPECT(call, code)                                                          \
    do {                                                                            \
        long long got_ = (long long)(call);                                         \
        if (got_ != (long long)(code)) {                                            \
            printf("FAIL line %d: got %lld, want %lld\n", __LINE__, got_,           \
                   (long long)(code));                                              \
            return 1;                                                               \
        }                                                                           \
    } while (0)

int main(void)
{
    char* a = (char*)(uintptr_t)0x100000;       /* aligned fake device addresses */
    const ptrdiff_t far = (ptrdiff_t)1 << 30;
    float* g = (float*)(a + 5 * far);
    dit_attn_args args = {2, 16, 32, 8, 4, 128, 0, QKR_BF16, 0.1f, NULL};
    dit_attn_tensor q, k, v, o, none = {NULL, 0, 0, 0};
    qkr_grad_tensor t;

    q.data = a, q.batch_stride = 16 * 1024, q.token_stride = 1024, q.head_stride = 128;
    k.data = a + far, k.batch_stride = 32 * 512, k.token_stride = 512, k.head_stride = 128;
    v = k, v.data = a + 2 * far;
    o = q, o.data = a + 3 * far;
    EXPECT(dit_attention_workspace_size(&args), 0);
    EXPECT(dit_attention(&args, &q, &k, &v, &o, NULL, NULL, 0, NULL), QKR_ERR_NULL);
    EXPECT(dit_attention(&args, &none, &k, &v, &o, g, NULL, 0, NULL), QKR_ERR_NULL);
    EXPECT(dit_attention(&args, &q, &k, &v, &q, g, NULL, 0, NULL), QKR_ERR_ARG);
    EXPECT(dit_attention_backward(&args, &o, &q, &k, &v, &o, g, &none, &k, &v, NULL, 0, NULL),
           QKR_ERR_NULL);
    args.head_dim = 80;
    EXPECT(dit_attention(&args, &q, &k, &v, &o, g, NULL, 0, NULL), QKR_ERR_UNSUPPORTED);
    args.head_dim = 128, args.batch = 0;
    EXPECT(dit_attention(&args, &q, &k, &v, &o, g, NULL, 0, NULL), QKR_OK);
    EXPECT(dit_attention(NULL, &q, &k, &v, &o, g, NULL, 0, NULL), QKR_ERR_NULL);

    EXPECT(dit_layer_norm(a, a + far, 0, 64, NULL, NULL, QKR_FP32, 1e-6f, QKR_BF16, NULL), QKR_OK);
    EXPECT(dit_layer_norm(a, a + 16, 4, 64, NULL, NULL, QKR_FP32, 1e-6f, QKR_BF16, NULL), QKR_ERR_ARG);
    EXPECT(dit_layer_norm(a, a + far, 4, DIT_LN_MAX_HIDDEN + 8, NULL, NULL, QKR_FP32, 1e-6f, QKR_BF16,
                          NULL), QKR_ERR_UNSUPPORTED);
    EXPECT(dit_layer_norm_backward_workspace_size(4, 60, 4), QKR_ERR_UNSUPPORTED);
    EXPECT(dit_layer_norm_backward(a, a + far, a + 2 * far, 4, 64, 4, NULL, DIT_LN_ONE_PLUS + 1, QKR_FP32,
                                   NULL, NULL, 1e-6f, QKR_BF16, NULL, 0, NULL), QKR_ERR_ARG);
    EXPECT(dit_layer_norm_backward(a, a + far, a + 2 * far, 4, 64, 4, NULL, DIT_LN_WEIGHT, QKR_FP32, g,
                                   NULL, 1e-6f, QKR_BF16, NULL, 0, NULL), QKR_ERR_NULL);

    t.grad = a, t.x = a + far, t.out = a;
    EXPECT(qknorm_rope_backward_workspace_size(100, 64), 50 * 2 * 64 * 4);
    EXPECT(qknorm_rope_backward(&t, &t, NULL, 4, 2, 64, g, g, g, g, 1e-6f, a, a, QKR_COS_SHARED, QKR_FP32,
                                QKR_ROPE_INTERLEAVED, QKR_BF16, NULL, 0, NULL), QKR_ERR_MODE);
    EXPECT(qknorm_rope_backward(&t, NULL, NULL, 4, 2, 64, g, g, g, NULL, 1e-6f, a, a, QKR_COS_SHARED,
                                QKR_FP32, QKR_ROPE_INTERLEAVED, QKR_BF16, NULL, 0, NULL), QKR_ERR_NULL);
    EXPECT(qknorm_rope_backward(&t, NULL, NULL, 4, 2, 64, g, g, g, g, 1e-6f, a, a, QKR_COS_SHARED,
                                QKR_FP32, QKR_ROPE_INTERLEAVED, QKR_BF16, NULL, 0, NULL),
           QKR_ERR_WORKSPACE);
    printf("ok\n");
    return 0;
}
