// layer_norm.hip -- layer norm forward and backward for gfx950 (see
// layer_norm.h).
//
// Bound by memory: every pass reads each row once and keeps it in registers.
// Forward 5.0 TB/s on 32760 x 5120, a large copy's rate on that card, where
// fuse_scale_shift, a wave a row, moves the same bytes at 6.0: the rest is the
// schedule's (two rows of a workgroup in flight, two reductions through LDS a row).
//   * a row is held by TPR threads, VPT 16-byte vectors each: one wave up to
//     1024 columns, the four waves of a workgroup above;
//   * a workgroup walks a run of rows of one weight row, so the weight (and in
//     the backward pass the sums of dweight and dbias) stay in registers, and
//     the loads of the next row are in flight while the present one is reduced;
//   * two reductions a row: sum x, then the squared deviations (forward) or
//     those with sum g and sum g (x - mean) (backward);
//   * the workgroups' sums of dweight and dbias go to the workspace and a
//     second kernel adds them in order: no atomics.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "layer_norm.h"
#include "norm_rows.h"

namespace {

using namespace qkr_dev;
using namespace qkr_rows;
using qkr_host::aligned16;
using qkr_host::overlaps;

struct LnParams {
    const uint16_t* x;
    const uint16_t* dy;
    uint16_t* out;             // y, or dx
    const void* weight;
    const void* bias;
    float* dweight;            // [batches][hidden], or NULL
    float* dbias;
    float* parts;              // [batches][chunks][2][hidden], when chunks > 1
    int64_t rows;
    uint32_t rows_per_batch;   // at most rows
    uint32_t chunks;           // workgroups of one batch
    uint32_t rows_per_chunk;
    int32_t hidden;
    int32_t param_dtype;
    float one;                 // added to the weight
    float eps;
};

// A row's mean, 1 / sqrt(var + eps) and, in the backward pass, sum g and
// sum g (x - mean), all of x * 2^-shift.  shift is 0 unless the plain sums
// leave fp32's range (16-bit values beyond about 1e17, or squares that sink
// into the subnormals while eps is as small): then it is the binary exponent
// of the row's largest |x|, an exact scaling.  rstd_x is 1 / sqrt(var + eps) of
// x itself, the factor of dx: at most 1 / sqrt(eps), so it is always finite,
// which rstd of a scaled row need not be (eps 2^-2shift may sink to 0).
struct RowStats {
    float mean, rstd, rstd_x, g, gd;
    int shift;
};

template <int TPR, int VPT, bool F16, bool GRAD, bool SCALED>
__device__ __forceinline__ RowStats plain_stats(const u32x4 (&x)[VPT], const u32x4 (&dy)[VPT],
                                                const float (&w)[VPT][8], int t, int nvec, int hidden,
                                                float eps, int shift, float* slot, float& ss)
{
    RowStats s;
    s.shift = shift;
    float sum[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        float f[8];
        unpack8<F16>(x[u], f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum[0] += SCALED ? __builtin_amdgcn_ldexpf(f[k], -shift) : f[k];
    }
    row_sums<TPR>(sum, slot);
    forget_unpacked(x);
    s.mean = sum[0] / (float)hidden;
    float v[GRAD ? 3 : 1] = {};
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        if (u * TPR + t < nvec) {
            float f[8], d[8];
            unpack8<F16>(x[u], f);
            if constexpr (GRAD)
                unpack8<F16>(dy[u], d);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float e = (SCALED ? __builtin_amdgcn_ldexpf(f[k], -shift) : f[k]) - s.mean;
                v[0] = __builtin_fmaf(e, e, v[0]);
                if constexpr (GRAD) {
                    const float g = d[k] * w[u][k];
                    v[1] += g;
                    v[2] = __builtin_fmaf(g, e, v[2]);
                }
            }
        }
    }
    row_sums<TPR>(v, slot + 4);
    forget_unpacked(x);
    forget_unpacked(dy);
    ss = v[0];
    s.rstd = ss / (float)hidden + eps;
    if constexpr (GRAD) {
        s.g = v[1];
        s.gd = v[2];
    }
    return s;
}

template <int TPR, int VPT, bool F16, bool GRAD>
__device__ __forceinline__ RowStats row_stats(const u32x4 (&x)[VPT], const u32x4 (&dy)[VPT],
                                              const float (&w)[VPT][8], int t, int nvec, int hidden,
                                              float eps, float* slot)
{
    float ss;
    RowStats s = plain_stats<TPR, VPT, F16, GRAD, false>(x, dy, w, t, nvec, hidden, eps, 0, slot, ss);
    // sum g (x - mean) may leave the range where its factors do not
    if (__builtin_expect(s.rstd <= 0x1.fffffep127f && (ss >= kTinySum || eps >= kTinySum) &&
                             (!GRAD || fabsf(s.gd) <= 0x1.fffffep127f), 1)) {
        s.rstd = s.rstd_x = __builtin_amdgcn_rsqf(s.rstd);
        return s;
    }
    float m = 0.0f;            // the same branch in every thread of the row
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        float f[8];
        unpack8<F16>(x[u], f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            m = fmaxf(m, fabsf(f[k]));
    }
    const int e = __builtin_amdgcn_frexp_expf(row_max<TPR>(m, slot));
    const float eps_s = __builtin_amdgcn_ldexpf(eps, -2 * e);
    if (!(eps_s <= 0x1.fffffep127f)) {
        // the variance is below eps by more than 2^128
        s.rstd = s.rstd_x = rsqrt_full_range(eps);
        return s;
    }
    s = plain_stats<TPR, VPT, F16, GRAD, true>(x, dy, w, t, nvec, hidden, eps_s, e, slot, ss);
    // a constant row of large values: eps 2^-2e may underflow to 0.  Any finite
    // rstd gives its n, which is exactly 0 (sums of up to 8192 equal 16-bit
    // values do not round), but not its dx.
    s.rstd = __builtin_amdgcn_rsqf(fmaxf(s.rstd, 0x1p-126f));
    s.rstd_x = ss == 0.0f ? rsqrt_full_range(eps) : __builtin_amdgcn_ldexpf(s.rstd, -e);
    return s;
}

// A workgroup's rows: TPR == 64 takes 4 at a time, one a wave.
template <int TPR, int VPT, bool F16, bool GRAD>
__global__ __launch_bounds__(kThreads, GRAD || VPT == 4 ? 2 : 3)
void layer_norm_kernel(const LnParams p)
{
    constexpr int RPW = kThreads / TPR;
    __shared__ __attribute__((aligned(16))) float slot[RPW == 1 ? 16 : 4];
    extern __shared__ float joined[];       // GRAD, RPW > 1: [3][2][hidden]
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int nvec = p.hidden / kVec;
    const uint32_t batch = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    const int64_t begin = (int64_t)batch * p.rows_per_batch;
    const int64_t batch_end = begin + p.rows_per_batch < p.rows ? begin + p.rows_per_batch : p.rows;
    const int64_t first = begin + (int64_t)chunk * p.rows_per_chunk;
    const int64_t end = first + p.rows_per_chunk < batch_end ? first + p.rows_per_chunk : batch_end;

    float w[VPT][8], b[GRAD ? 1 : VPT][8], dw[GRAD ? VPT : 1][8], db[GRAD ? VPT : 1][8];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int i = u * TPR + t;
        const bool there = i < nvec;
        if (p.weight && there) {
            load_params(p.weight, (int64_t)batch * p.hidden + i * kVec, p.param_dtype, w[u]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[u][k] += p.one;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[u][k] = 1.0f;
        }
        if constexpr (GRAD) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                dw[u][k] = db[u][k] = 0.0f;
        } else {
            if (p.bias && there) {
                load_params(p.bias, i * kVec, p.param_dtype, b[u]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    b[u][k] = 0.0f;
            }
        }
    }

    u32x4 x[VPT], dy[VPT], nx[VPT], ndy[VPT];
    const auto fetch = [&](int64_t r) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = u * TPR + t;
            nx[u] = ndy[u] = u32x4{0, 0, 0, 0};
            if (r < end && i < nvec) {
                nx[u] = load16<true>(p.x + r * p.hidden + i * kVec);
                if constexpr (GRAD)
                    ndy[u] = load16<true>(p.dy + r * p.hidden + i * kVec);
            }
        }
    };
    fetch(first + sub);
    for (int64_t r = first + sub; r < end; r += RPW) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            x[u] = nx[u];
            dy[u] = ndy[u];
        }
        fetch(r + RPW);
        const RowStats s = row_stats<TPR, VPT, F16, GRAD>(x, dy, w, t, nvec, p.hidden, p.eps, slot);
        const float c1 = s.g / (float)p.hidden;
        const float c2 = s.gd * s.rstd / (float)p.hidden;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
                float f[8], d[8], o[8];
                unpack8<F16>(x[u], f);
                if constexpr (GRAD)
                    unpack8<F16>(dy[u], d);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float e = s.shift ? __builtin_amdgcn_ldexpf(f[k], -s.shift) : f[k];
                    const float n = (e - s.mean) * s.rstd;
                    if constexpr (GRAD) {
                        o[k] = __builtin_fmaf(-n, c2, __builtin_fmaf(d[k], w[u][k], -c1)) * s.rstd_x;
                        dw[u][k] = __builtin_fmaf(d[k], n, dw[u][k]);
                        db[u][k] += d[k];
                    } else {
                        o[k] = __builtin_fmaf(n, w[u][k], b[u][k]);
                    }
                }
                store16<true>(p.out + r * p.hidden + i * kVec, pack8<F16>(o));
            }
        }
    }

    if constexpr (GRAD) {
        if (!p.dweight)
            return;
        if constexpr (RPW > 1) {            // the four waves' sums, in wave order
            if (sub > 0) {
#pragma unroll
                for (int u = 0; u < VPT; ++u) {
                    const int i = u * TPR + t;
                    if (i < nvec) {
                        float* at = joined + (sub - 1) * 2 * p.hidden + i * kVec;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            at[k] = dw[u][k];
                            at[p.hidden + k] = db[u][k];
                        }
                    }
                }
            }
            __syncthreads();
            if (sub > 0)
                return;
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int i = u * TPR + t;
                if (i < nvec) {
                    for (int j = 0; j < RPW - 1; ++j) {
                        const float* at = joined + j * 2 * p.hidden + i * kVec;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            dw[u][k] += at[k];
                            db[u][k] += at[p.hidden + k];
                        }
                    }
                }
            }
        }
        float* wo = p.dweight + (int64_t)batch * p.hidden;
        float* bo = p.dbias + (int64_t)batch * p.hidden;
        if (p.chunks > 1) {
            wo = p.parts + (int64_t)blockIdx.x * 2 * p.hidden;
            bo = wo + p.hidden;
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
                f32x4* a = reinterpret_cast<f32x4*>(wo + i * kVec);
                f32x4* c = reinterpret_cast<f32x4*>(bo + i * kVec);
                a[0] = f32x4{dw[u][0], dw[u][1], dw[u][2], dw[u][3]};
                a[1] = f32x4{dw[u][4], dw[u][5], dw[u][6], dw[u][7]};
                c[0] = f32x4{db[u][0], db[u][1], db[u][2], db[u][3]};
                c[1] = f32x4{db[u][4], db[u][5], db[u][6], db[u][7]};
            }
        }
    }
}

// dweight and dbias of a batch: the sums of its chunks' parts.  16 threads
// side by side hold 4 columns each, 16 such rows take every 16th part.
__global__ __launch_bounds__(kThreads)
void layer_norm_parts_kernel(const LnParams p)
{
    __shared__ f32x4 sums[16][16];
    const int cols = 2 * p.hidden, per = (cols + 63) / 64;
    const uint32_t batch = blockIdx.x / per;
    const int col = (int)(blockIdx.x % per) * 64 + threadIdx.x % 16 * 4, row = threadIdx.x / 16;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < cols) {
        const float* at = p.parts + (int64_t)batch * p.chunks * cols + col;
#pragma unroll 8
        for (uint32_t i = row; i < p.chunks; i += 16)
            s += *reinterpret_cast<const f32x4*>(at + (int64_t)i * cols);
    }
    sums[row][threadIdx.x % 16] = s;
    __syncthreads();
    if (row == 0 && col < cols) {
#pragma unroll
        for (int i = 1; i < 16; ++i)
            s += sums[i][threadIdx.x];
        float* to = col < p.hidden ? p.dweight + (int64_t)batch * p.hidden + col
                                   : p.dbias + (int64_t)batch * p.hidden + col - p.hidden;
        *reinterpret_cast<f32x4*>(to) = s;
    }
}

// One wave a row up to this width, the whole workgroup above it.
constexpr int kWaveHidden = 1024;

// Vectors a thread holds of a row (the kernels' VPT).
int vectors_of(int hidden)
{
    const int nvec = hidden / kVec, threads = hidden <= kWaveHidden ? kWave : kThreads;
    return (nvec + threads - 1) / threads;
}

using Fn = void (*)(LnParams);

template <bool F16, bool GRAD>
Fn select(int hidden)
{
    const int v = vectors_of(hidden);
    if (hidden <= kWaveHidden)
        return v == 1 ? layer_norm_kernel<64, 1, F16, GRAD> : layer_norm_kernel<64, 2, F16, GRAD>;
    switch (v) {
    case 1: return layer_norm_kernel<256, 1, F16, GRAD>;
    case 2: return layer_norm_kernel<256, 2, F16, GRAD>;
    case 3: return layer_norm_kernel<256, 3, F16, GRAD>;
    default: return layer_norm_kernel<256, 4, F16, GRAD>;
    }
}

// Workgroups that a call spreads its rows over, by the vectors a thread holds:
// with one of them, as many as keep enough loads in flight; with more, a whole
// multiple of what the registers let run at once, where that is 2 or 3 a CU (the
// last round is then as full as the others).  Measured on 300 MB of rows, in
// workgroups a CU (GB/s; * the rule's):
//   forward   512 columns (a wave a row, 1 vector): 2: 3645, 3: 4421, 4: 5048*
//            1024 (a wave a row, 2 vectors):        2: 4975, 3: 4706, 4: 5073*
//            2048 (1 vector):                       2: 3000, 3: 4101, 4: 4809*
//            4096 (2 vectors):                      2: 4780, 3: 4690, 4: 5082*
//            5120 (3 vectors):                      2: 4717, 3: 5044*, 4: 4223
//            6144 (3 vectors, the last one full):   2: 5014, 3: 4686*, 4: 4431
//            8192 (4 vectors):                      2: 5163, 3: 4271, 4: 5265*
//   backward  512 columns (a wave a row, 1 vector): 2: 4271, 3: 4569, 4: 4812*
//            1024 (a wave a row, 2 vectors):        2: 4946*, 3: 4651, 4: 4470
//            2048 (1 vector):                       2: 3627, 3: 4323, 4: 4610*
//            4096 (2 vectors):                      2: 4908*, 3: 4515, 4: 4108
//            5120 (3 vectors):                      2: 4892*, 3: 3994, 4: 4486
//            6144 (3 vectors, the last one full):   2: 4760*, 3: 4052, 4: 4731
//            8192 (4 vectors):                      2: 4697*, 3: 3993, 4: 4647
int64_t target_blocks(int hidden, bool grad)
{
    const int v = vectors_of(hidden);
    return 256 * (grad ? (v == 1 ? 4 : 2) : (v == 3 ? 3 : 4));
}

// Workgroups a batch: its rows spread so that the whole call has about
// target_blocks() of them, none without a row.
int64_t chunks_of(int64_t rows, int hidden, int64_t rows_per_batch, bool grad)
{
    const int64_t per = rows_per_batch < rows ? rows_per_batch : rows;
    const int64_t batches = (rows + per - 1) / per;
    const int64_t at_once = hidden <= kWaveHidden ? 4 : 1;
    const int64_t most = (per + at_once - 1) / at_once;
    int64_t chunks = target_blocks(hidden, grad) / batches;
    chunks = chunks < 1 ? 1 : chunks < most ? chunks : most;
    const int64_t each = ((per + chunks - 1) / chunks + at_once - 1) / at_once * at_once;
    return (per + each - 1) / each;
}

int check_sizes(int64_t rows, int32_t hidden, int64_t rows_per_batch)
{
    if (hidden < kVec || hidden > DIT_LN_MAX_HIDDEN || hidden % kVec)
        return QKR_ERR_UNSUPPORTED;
    if (rows < 0 || rows >= QKR_MAX_TOKENS || rows_per_batch < 1)
        return QKR_ERR_SHAPE;
    return QKR_OK;
}

// Weight rows that the rows use; rows_per_batch may be any size.
int64_t batches_of(int64_t rows, int64_t rows_per_batch)
{
    return rows / rows_per_batch + (rows % rows_per_batch != 0);
}

int check_types(int32_t dtype, int32_t param_dtype, float eps)
{
    if (dtype < QKR_BF16 || dtype > QKR_FP32 || param_dtype < QKR_BF16 || param_dtype > QKR_FP32)
        return QKR_ERR_ARG;
    if (dtype == QKR_FP32)
        return QKR_ERR_UNSUPPORTED;
    return eps > 0.0f && isfinite(eps) ? QKR_OK : QKR_ERR_ARG;
}

void fill(LnParams& p, int64_t rows, int hidden, int64_t rows_per_batch, bool grad)
{
    p.rows = rows;
    p.hidden = hidden;
    p.rows_per_batch = (uint32_t)(rows_per_batch < rows ? rows_per_batch : rows);
    p.chunks = (uint32_t)chunks_of(rows, hidden, rows_per_batch, grad);
    const uint32_t at_once = hidden <= kWaveHidden ? 4 : 1;
    p.rows_per_chunk = ((p.rows_per_batch + p.chunks - 1) / p.chunks + at_once - 1) / at_once * at_once;
}

hipError_t launch(Fn fn, int64_t blocks, size_t lds, LnParams& p, void* stream)
{
    void* args[] = {&p};
    return hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)blocks), dim3(kThreads),
                           args, lds, static_cast<hipStream_t>(stream));
}

}  // namespace

extern "C" int dit_layer_norm(const void* x, void* y, int64_t rows, int32_t hidden,
                              const void* weight, const void* bias, int32_t param_dtype, float eps,
                              int32_t dtype, void* stream)
{
    int rc = check_types(dtype, param_dtype, eps);
    if (rc == QKR_OK)
        rc = check_sizes(rows, hidden, 1);
    if (rc != QKR_OK || rows == 0)
        return rc;
    if (!x || !y)
        return QKR_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(weight) || !aligned16(bias))
        return QKR_ERR_ALIGN;
    const uint64_t bytes = (uint64_t)rows * (uint64_t)hidden * 2u;
    const uint64_t param_bytes = (uint64_t)hidden * (param_dtype == QKR_FP32 ? 4u : 2u);
    if ((x != y && overlaps(x, bytes, y, bytes)) ||
        overlaps(y, bytes, weight, weight ? param_bytes : 0) ||
        overlaps(y, bytes, bias, bias ? param_bytes : 0))
        return QKR_ERR_ARG;
    LnParams p = {};
    p.x = static_cast<const uint16_t*>(x);
    p.out = static_cast<uint16_t*>(y);
    p.weight = weight;
    p.bias = bias;
    p.param_dtype = param_dtype;
    p.eps = eps;
    fill(p, rows, hidden, rows, false);
    Fn fn = dtype == QKR_FP16 ? select<true, false>(hidden) : select<false, false>(hidden);
    return launch(fn, p.chunks, 0, p, stream) == hipSuccess ? QKR_OK : QKR_ERR_HIP;
}

extern "C" int64_t dit_layer_norm_backward_workspace_size(int64_t rows, int32_t hidden,
                                                          int64_t rows_per_batch)
{
    const int rc = check_sizes(rows, hidden, rows_per_batch);
    if (rc != QKR_OK || rows == 0)
        return rc;
    const int64_t chunks = chunks_of(rows, hidden, rows_per_batch, true);
    const int64_t batches = batches_of(rows, rows_per_batch);
    return chunks == 1 ? 0 : batches * chunks * 2 * hidden * 4;
}

extern "C" int dit_layer_norm_backward(const void* dy, const void* x, void* dx, int64_t rows,
                                       int32_t hidden, int64_t rows_per_batch, const void* weight,
                                       int32_t weight_form, int32_t param_dtype, float* dweight,
                                       float* dbias, float eps, int32_t dtype, void* workspace,
                                       int64_t workspace_bytes, void* stream)
{
    int rc = check_types(dtype, param_dtype, eps);
    if (rc == QKR_OK && weight_form != DIT_LN_WEIGHT && weight_form != DIT_LN_ONE_PLUS)
        rc = QKR_ERR_ARG;
    if (rc == QKR_OK)
        rc = check_sizes(rows, hidden, rows_per_batch);
    if (rc != QKR_OK || rows == 0)
        return rc;
    if (!dy || !x || !dx || !dweight != !dbias)
        return QKR_ERR_NULL;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(dx) || !aligned16(weight) ||
        !aligned16(dweight) || !aligned16(dbias))
        return QKR_ERR_ALIGN;
    const int64_t need = dweight ? dit_layer_norm_backward_workspace_size(rows, hidden, rows_per_batch)
                                 : 0;
    if (need && (!workspace || workspace_bytes < need))
        return QKR_ERR_WORKSPACE;
    if (need && !aligned16(workspace))
        return QKR_ERR_ALIGN;
    const uint64_t bytes = (uint64_t)rows * (uint64_t)hidden * 2u;
    const uint64_t params = (uint64_t)batches_of(rows, rows_per_batch) * (uint64_t)hidden;
    const struct { const void* at; uint64_t n; } in[] = {
        {dy, bytes}, {x, bytes}, {weight, weight ? params * (param_dtype == QKR_FP32 ? 4u : 2u) : 0}};
    const struct { const void* at; uint64_t n; } out[] = {
        {dx, bytes}, {dweight, dweight ? params * 4 : 0}, {dbias, dbias ? params * 4 : 0},
        {workspace, (uint64_t)need}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j)
            if (!(i == 0 && j == 0 && dx == dy) && overlaps(out[i].at, out[i].n, in[j].at, in[j].n))
                return QKR_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].at, out[i].n, out[j].at, out[j].n))
                return QKR_ERR_ARG;
    }
    LnParams p = {};
    p.x = static_cast<const uint16_t*>(x);
    p.dy = static_cast<const uint16_t*>(dy);
    p.out = static_cast<uint16_t*>(dx);
    p.weight = weight;
    p.param_dtype = param_dtype;
    p.one = weight_form == DIT_LN_ONE_PLUS ? 1.0f : 0.0f;
    p.dweight = dweight;
    p.dbias = dbias;
    p.parts = static_cast<float*>(workspace);
    p.eps = eps;
    fill(p, rows, hidden, rows_per_batch, true);
    const int64_t batches = batches_of(rows, rows_per_batch);
    Fn fn = dtype == QKR_FP16 ? select<true, true>(hidden) : select<false, true>(hidden);
    const size_t lds = dweight && hidden <= kWaveHidden ? (size_t)3 * 2 * hidden * 4 : 0;
    hipError_t err = launch(fn, batches * p.chunks, lds, p, stream);
    if (err == hipSuccess && dweight && p.chunks > 1)
        err = launch(layer_norm_parts_kernel, batches * ((2 * hidden + 63) / 64), 0, p, stream);
    return err == hipSuccess ? QKR_OK : QKR_ERR_HIP;
}
