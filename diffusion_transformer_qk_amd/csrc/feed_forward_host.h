// feed_forward_host.h -- argument checks and tile choice shared by the gated
// feed-forward entry points.  Internal header.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "feed_forward.h"
#include "host_common.h"

namespace qkr_ff_host {

inline int check_args(const dit_ff_args* a, bool forward)
{
    if (!a)
        return QKR_ERR_NULL;
    const bool fp8 = a->dtype == DIT_FF_E4M3;
    if ((!fp8 && (a->dtype < QKR_BF16 || a->dtype > QKR_FP32)) || a->out_dtype < QKR_BF16 ||
        a->out_dtype > QKR_FP32 || (a->activation != DIT_FF_SILU && a->activation != DIT_FF_GELU_TANH))
        return QKR_ERR_ARG;
    if (a->dtype == QKR_FP32 || a->out_dtype == QKR_FP32 || (fp8 && !forward))
        return QKR_ERR_UNSUPPORTED;
    if (!fp8 && a->out_dtype != a->dtype)
        return QKR_ERR_ARG;
    const int unit = fp8 ? 16 : 8;
    if (a->hidden < unit || a->inner < unit || a->hidden % unit || a->inner % unit ||
        a->hidden > DIT_FF_MAX_WIDTH || a->inner > DIT_FF_MAX_WIDTH)
        return QKR_ERR_UNSUPPORTED;
    // a launch holds fewer than 2^32 work-items, a workgroup 256 for 128 x 128 outputs
    if (a->rows < 0 || a->rows >= QKR_MAX_TOKENS ||
        (a->rows / 128 + 1) * (a->inner / 64 + 2) >= ((int64_t)1 << 24) ||
        (a->rows / 128 + 1) * (a->hidden / 64 + 2) >= ((int64_t)1 << 24))
        return QKR_ERR_SHAPE;
    return QKR_OK;
}

struct Buffer {
    const void* at;
    uint64_t bytes;
    uintptr_t align;
};

// Alignment of all, and whether an output meets another buffer.
inline int check_buffers(const Buffer* in, int ins, const Buffer* out, int outs)
{
    for (int i = 0; i < ins; ++i)
        if (reinterpret_cast<uintptr_t>(in[i].at) & (in[i].align - 1))
            return QKR_ERR_ALIGN;
    for (int i = 0; i < outs; ++i)
        if (reinterpret_cast<uintptr_t>(out[i].at) & (out[i].align - 1))
            return QKR_ERR_ALIGN;
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < ins; ++j)
            if (qkr_host::overlaps(out[i].at, out[i].bytes, in[j].at, in[j].bytes))
                return QKR_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (qkr_host::overlaps(out[i].at, out[i].bytes, out[j].at, out[j].bytes))
                return QKR_ERR_ARG;
    }
    return QKR_OK;
}

// Whether a product of `rows` x `columns` outputs is cut into 256 x 256 tiles
// (one workgroup a CU) rather than 128 x 128 (two a CU).
inline bool large_tiles(int64_t rows, int64_t columns)
{
    return (rows + 255) / 256 * ((columns + 255) / 256) >= 256;
}

template <typename Params>
inline int launch(void (*fn)(Params), int64_t blocks, Params& p, void* stream, unsigned threads = 256)
{
    void* args[] = {&p};
    return hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)blocks), dim3(threads), args, 0,
                           static_cast<hipStream_t>(stream)) == hipSuccess
               ? QKR_OK
               : QKR_ERR_HIP;
}

}  // namespace qkr_ff_host
