// attention_host.h -- argument checks shared by the attention entry points.
// Internal header.
#pragma once

#include <math.h>
#include <stdint.h>

#include "dit_attention.h"
#include "host_common.h"

namespace qkr_attn_host {

struct Extent {
    int64_t tokens;
    int32_t heads;
};

struct Range {
    const void* at;
    uint64_t bytes;
};

// Workgroups of one launch, and rows of one sample's head group, stay below
// these (a launch holds fewer than 2^32 work-items; row numbers are 32-bit).
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;

inline int check_args(const dit_attn_args* a)
{
    if (!a)
        return QKR_ERR_NULL;
    if (a->dtype < QKR_BF16 || a->dtype > QKR_FP32 || (a->causal != 0 && a->causal != 1) ||
        !isfinite(a->scale * 1.5f) || !(a->scale > 0.0f))      // it is used times log2(e)
        return QKR_ERR_ARG;
    if (a->dtype == QKR_FP32 || (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256))
        return QKR_ERR_UNSUPPORTED;
    if (a->batch < 0 || a->q_tokens < 0 || a->kv_tokens < 0 || a->q_tokens >= QKR_MAX_TOKENS ||
        a->kv_tokens >= QKR_MAX_TOKENS || a->batch >= QKR_MAX_TOKENS || a->kv_heads < 1 ||
        a->heads < a->kv_heads || a->heads > QKR_MAX_HEADS || a->heads % a->kv_heads)
        return QKR_ERR_SHAPE;
    // tokens are dealt to workgroups in blocks of 32 or more
    if (a->q_tokens * (a->heads / a->kv_heads) >= kMaxRows ||
        a->batch * a->heads * (a->q_tokens / 32 + 1) >= kMaxBlocks ||
        a->batch * a->kv_heads * (a->kv_tokens / 32 + 1) >= kMaxBlocks)
        return QKR_ERR_SHAPE;
    return QKR_OK;
}

// A call's tensor as the checks and kernels take it: the strides of dimensions
// of one element, which may be anything, replaced by some that fit (0, and for a
// token at least head_dim: what kernels stage past the last token lies outside
// the buffer's range, and reads as zero, only if its rows are a row apart).  One
// without tokens may be NULL.
inline dit_attn_tensor plain(const dit_attn_args& a, const dit_attn_tensor* t, const Extent& e)
{
    dit_attn_tensor p = t ? *t : dit_attn_tensor{};
    if (a.batch == 1)
        p.batch_stride = 0;
    if (e.tokens <= 1)
        p.token_stride = a.head_dim;
    if (e.heads == 1)
        p.head_stride = 0;
    return p;
}

// Elements from the first to one past the last of a tensor.
inline uint64_t span(const dit_attn_args& a, const dit_attn_tensor& t, const Extent& e)
{
    if (e.tokens == 0)
        return 0;
    return (uint64_t)(a.batch - 1) * t.batch_stride + (uint64_t)(e.tokens - 1) * t.token_stride +
           (uint64_t)(e.heads - 1) * t.head_stride + a.head_dim;
}

inline Range range(const dit_attn_args& a, const dit_attn_tensor& t, const Extent& e)
{
    return e.tokens ? Range{t.data, span(a, t, e) * 2} : Range{nullptr, 0};
}

inline bool meet(const Range& x, const Range& y) { return qkr_host::overlaps(x.at, x.bytes, y.at, y.bytes); }

// Whether two elements of the tensor share memory, or may: each dimension,
// smallest stride first, has to step past all that the smaller ones cover.
inline bool overlaps_itself(const dit_attn_args& a, const dit_attn_tensor& t, const Extent& e)
{
    struct { int64_t n, s; } dim[3] = {{a.batch, t.batch_stride}, {e.tokens, t.token_stride},
                                       {e.heads, t.head_stride}};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (dim[j].s > dim[j + 1].s) {
                const auto x = dim[j];
                dim[j] = dim[j + 1];
                dim[j + 1] = x;
            }
    int64_t covered = a.head_dim;
    for (const auto& d : dim)
        if (d.n > 1) {
            if (d.s < covered)
                return true;
            covered += (d.n - 1) * d.s;
        }
    return false;
}

inline int check_tensor(const dit_attn_args& a, const dit_attn_tensor& t, const Extent& e, bool written)
{
    if (e.tokens == 0)
        return QKR_OK;
    if (!t.data)
        return QKR_ERR_NULL;
    if (!qkr_host::aligned16(t.data) || t.batch_stride % 8 || t.token_stride % 8 ||
        t.head_stride % 8)
        return QKR_ERR_ALIGN;
    // more than the card holds, and batch * heads < 2^23 (check_args) keeps a
    // span in bytes inside 64 bits
    constexpr int64_t kMax = (int64_t)1 << 38;
    if (t.batch_stride < 0 || t.token_stride < 0 || t.head_stride < 0 || t.batch_stride > kMax ||
        t.head_stride > kMax || t.token_stride > DIT_ATTN_MAX_TOKEN_STRIDE ||
        t.token_stride < a.head_dim)
        return QKR_ERR_SHAPE;
    return written && overlaps_itself(a, t, e) ? QKR_ERR_ARG : QKR_OK;
}

// One dimension of two tensors that step through it alike: the stride, and each
// one's number of steps.
struct Steps {
    int64_t stride, x, y;
};

// Whether, of two tensors whose elements are runs of `width` at the steps of n
// dimensions (largest stride first), y's first run `ahead` of x's, two runs
// meet: whether the steps' difference can bring `ahead` within a run.  Along one
// dimension only a few differences can, unless its stride is far below what the
// smaller ones cover: then this says yes without looking.
inline bool runs_meet(int64_t ahead, const Steps* d, int n, int64_t width)
{
    if (n == 0)
        return -width < ahead && ahead < width;
    int64_t back = width - 1, forth = width - 1;     // what the smaller dimensions can take off or add
    for (int i = 1; i < n; ++i) {
        back += d[i].x * d[i].stride;
        forth += d[i].y * d[i].stride;
    }
    // ahead + k stride in [-forth, back], k in [-x, y]
    const auto floor_div = [](int64_t p, int64_t q) { return p / q - (p % q < 0); };
    int64_t first = -floor_div(forth + ahead, d->stride), last = floor_div(back - ahead, d->stride);
    first = first < -d->x ? -d->x : first;
    last = last > d->y ? d->y : last;
    if (last - first >= 16)
        return true;
    for (int64_t k = first; k <= last; ++k)
        if (runs_meet(ahead + k * d->stride, d + 1, n - 1, width))
            return true;
    return false;
}

// Whether two tensors may share an element.  Ranges that do not meet settle
// it; of tensors that interleave, slices of one buffer are told apart: those of
// the same strides whatever their order, and rows of the same token stride whose
// columns do not meet, at batch strides that are whole rows.
inline bool may_meet(const dit_attn_args& a, const dit_attn_tensor& x, const Extent& ex,
                     const dit_attn_tensor& y, const Extent& ey)
{
    if (ex.tokens == 0 || ey.tokens == 0 || !meet(range(a, x, ex), range(a, y, ey)))
        return false;
    const int64_t ahead =                                 // both are 16-byte aligned
        (reinterpret_cast<intptr_t>(y.data) - reinterpret_cast<intptr_t>(x.data)) / 2;
    const struct { int64_t nx, ny, sx, sy; } dims[] = {
        {a.batch, a.batch, x.batch_stride, y.batch_stride},
        {ex.tokens, ey.tokens, x.token_stride, y.token_stride},
        {ex.heads, ey.heads, x.head_stride, y.head_stride}};
    Steps steps[3];
    int n = 0;
    bool alike = true;
    for (const auto& d : dims) {
        const int64_t s = d.nx > 1 ? d.sx : d.sy;
        alike = alike && (d.nx == 1 || d.ny == 1 || d.sx == d.sy);
        if (s == 0 || (d.nx == 1 && d.ny == 1))           // a dimension that leads nowhere
            continue;
        int i = n++;
        for (; i > 0 && steps[i - 1].stride < s; --i)
            steps[i] = steps[i - 1];
        steps[i] = Steps{s, d.nx - 1, d.ny - 1};
    }
    if (alike && !runs_meet(ahead, steps, n, a.head_dim))
        return false;
    // rows: what tokens (or, of one token each, samples) step by
    int64_t ts = ex.tokens > 1 ? x.token_stride : y.token_stride;
    if (ex.tokens > 1 && ey.tokens > 1 && ts != y.token_stride)
        return true;
    if (ex.tokens == 1 && ey.tokens == 1)
        ts = x.batch_stride == 0 || (y.batch_stride != 0 && y.batch_stride < x.batch_stride) ? y.batch_stride
                                                                                            : x.batch_stride;
    if (ts == 0)
        return true;
    if (a.batch > 1 && (x.batch_stride % ts || y.batch_stride % ts))
        return true;
    const int64_t wx = (ex.heads - 1) * x.head_stride + a.head_dim;
    const int64_t wy = (ey.heads - 1) * y.head_stride + a.head_dim;
    const int64_t column = ahead % ts < 0 ? ahead % ts + ts : ahead % ts;   // where y's begin in x's rows
    return !(wx <= column && column + wy <= ts);
}

// A tensor's pointer and strides as a kernel takes them.
template <typename T>
inline void unpack(const dit_attn_tensor& t, T*& at, int64_t& bs, int64_t& ts, int64_t& hs)
{
    at = static_cast<T*>(t.data);
    bs = t.batch_stride;
    ts = t.token_stride;
    hs = t.head_stride;
}

}  // namespace qkr_attn_host
