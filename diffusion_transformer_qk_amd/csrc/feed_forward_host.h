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

// The 16-bit terms of dgate and dup in the products that use them.  With one, a gradient
// is off by 1.41 times its own rounding in the mean, but by up to 1.84 where few numbers
// are rounded (600 calls of 1 to 20000 rows: above 1.5 with up to 25 rows, or with up
// to 22000 numbers); with two by its own rounding alone.  Two cost calls of few rows
// little, as the weights' way bounds them (x of 5120, W of 13824: one row 168 and 171 us,
// 32 rows 173 and 180; 128 rows 198 and 255), and small ones a launch (32 rows of 96, 264
// columns: 18.6 and 21.9; 64 of 8192, 512: 26.0 and 31.9).
inline int terms_of(const dit_ff_args& a)
{
    const int64_t small = (int64_t)1 << 15;
    return a.rows <= 32 || (a.rows * a.inner <= small && a.rows * a.hidden <= 32 * small) ? 2 : 1;
}

// How a product of rows x columns outputs and `stages` stages of k is cut: tiles of
// 256 x 256 (a workgroup a CU) or of 128 x 128 (two a CU), and k into splits whose
// sums are added by a launch of their own.  The cheapest by what a stage of a round
// of workgroups takes, as measured: 1.5 us of the large tiles, 0.95 of the small ones
// and 0.6 where they have a CU each.  (x of 5120, W of 13824: 512 rows 125 us with
// large tiles, 156 with small ones; 256 rows 106 and 91.  dx of one row 242 us without
// splits and 52 with the 12 that this gives, of 256 rows 263 and 115; dw of 16384 rows,
// 512 x 2048, 188 and 116.)
struct Cut {
    bool large;
    int64_t splits;
    int64_t row_tiles, column_tiles;
};

inline Cut cut_of(int64_t rows, int64_t columns, int64_t stages, bool may_split)
{
    Cut best = {};
    double least = 0.0;
    for (int large = 0; large < 2; ++large) {
        const int64_t side = large ? 256 : 128;
        const int64_t row_tiles = (rows + side - 1) / side, column_tiles = (columns + side - 1) / side;
        const int64_t tiles = row_tiles * column_tiles;
        for (int64_t splits = 1; splits <= 32; ++splits) {
            if (splits > 1 && (!may_split || stages / splits < 8 || tiles * splits > 512))
                break;
            const int64_t blocks = tiles * splits, at_once = large ? 256 : 512;
            const int64_t rounds = (blocks + at_once - 1) / at_once, each = (stages + splits - 1) / splits;
            const double stage = large ? 1.5 : blocks <= 256 ? 0.6 : 0.95;
            // the launch that adds the splits, and their way through memory
            const double join = splits > 1 ? 5.0 + 8e-6 * (double)(splits * rows * columns) / 4.0 : 0.0;
            const double time = (double)rounds * (double)each * stage + join;
            if (best.row_tiles == 0 || time < least) {
                best = Cut{large != 0, splits, row_tiles, column_tiles};
                least = time;
            }
        }
    }
    return best;
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
