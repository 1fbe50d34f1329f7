// rms_norm.hip -- RMS norm with the residual's addition and an 8-bit output, and
// its backward pass, for gfx950 (see rms_norm.h).
//
// Bound by memory: every pass reads each row once and keeps it in registers,
// VPT 16-byte vectors a thread.
//   * forward: one wave a row up to 1024 columns, the four waves of a workgroup
//     above, one row each: few registers, so that eight workgroups a CU keep
//     loads in flight.  The sum of squares and, for 8 bits, the largest
//     |s weight| are one reduction: the values in 8 bits are t * (448 / top),
//     without the norm;
//     32760 rows of 5120 with a residual: 224 us, 6.0 TB/s (a large copy: 5.1);
//     8 rows to 8 bits: 4.7 us (the call takes the host 11);
//   * backward: a workgroup walks a run of rows, the weight and the sums of dweight
//     stay in registers, and the loads of the next row are in flight while the
//     present one is reduced.  The workgroups' sums go to the workspace and a
//     second kernel adds them in order: no atomics.  65520 rows of 5120 with the
//     sum's gradient: 516 and 5 us, 5.2 TB/s.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "norm_rows.h"
#include "rms_norm.h"

namespace {

using namespace qkr_dev;
using namespace qkr_rows;
using qkr_host::aligned16;
using qkr_host::overlaps;

constexpr float kMax = 0x1.fffffep127f;
constexpr float kFp8Max = 448.0f;

struct RmsParams {
    const uint16_t* x;         // s, in the backward pass
    const uint16_t* residual;  // dsum, in the backward pass
    const uint16_t* dy;
    uint16_t* sum;
    void* out;                 // y, or dx
    float* scales;
    const void* weight;
    float* dweight;            // [hidden], or NULL
    float* parts;              // [chunks][hidden], when chunks > 1
    int64_t rows;
    uint32_t chunks;           // workgroups of the backward pass
    uint32_t rows_per_chunk;
    int32_t hidden;
    int32_t param_dtype;
    float eps;
};

__device__ __forceinline__ void load_weight(const RmsParams& p, int i, bool there, float w[8])
{
    if (p.weight && there) {
        load_params(p.weight, i * kVec, p.param_dtype, w);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = 1.0f;
    }
}

__device__ __forceinline__ float scaled(float f, int shift) { return __builtin_amdgcn_ldexpf(f, -shift); }

// The sum of squares of a row's values times 2^-shift, and, with TOP, the
// largest of |value weight|.  `slot`: 8 floats of LDS.
template <int TPR, int VPT, bool F16, bool TOP, bool SCALED>
__device__ __forceinline__ void row_norm(const u32x4 (&x)[VPT], const RmsParams& p, int t, int nvec, int shift,
                                         float* slot, float& ss, float& top)
{
    float v[1] = {0.0f};
    top = 0.0f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        float f[8], w[8];
        unpack8<F16>(x[u], f);
        if constexpr (TOP)
            load_weight(p, u * TPR + t, u * TPR + t < nvec, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float e = SCALED ? scaled(f[k], shift) : f[k];
            v[0] = __builtin_fmaf(e, e, v[0]);
            if constexpr (TOP)
                top = fmaxf(top, fabsf(e * w[k]));
        }
    }
    if constexpr (TOP) {
        top = wave_max(top);
        if (TPR > kWave && threadIdx.x % kWave == 0)
            slot[4 + threadIdx.x / kWave] = top;
    }
    row_sums<TPR>(v, slot);
    if constexpr (TOP && TPR > kWave)
        top = fmaxf(fmaxf(slot[4], slot[5]), fmaxf(slot[6], slot[7]));
    ss = v[0];
}

// The row's largest |x|.
template <int TPR, int VPT, bool F16>
__device__ __forceinline__ float row_largest(const u32x4 (&x)[VPT], float* slot)
{
    float m = 0.0f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        float f[8];
        unpack8<F16>(x[u], f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            m = fmaxf(m, fabsf(f[k]));
    }
    return row_max<TPR>(m, slot);
}

__device__ __forceinline__ uint64_t fp8x8(const float (&o)[8])
{
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(o[0], o[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(o[2], o[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(o[4], o[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(o[6], o[7], hi, true);
    return (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo;
}

// s weight 2^-e: the product's mantissa is rounded as any product's is, whatever its
// exponent.
__device__ __forceinline__ float product(float s, float weight, int e)
{
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_frexp_mantf(s) * __builtin_amdgcn_frexp_mantf(weight),
                                   __builtin_amdgcn_frexp_expf(s) + __builtin_amdgcn_frexp_expf(weight) - e);
}

// A row to 8 bits whose largest |s weight| is too small for the products, or for 448
// over it: the values by product(), with the exponent of the largest.  s is read
// again, a vector at a time: held in registers it would cost the other rows theirs.
// rstd is of s 2^-shift.
template <int TPR, bool F16>
__device__ __forceinline__ void small_to_8_bits(const RmsParams& p, const uint16_t* s, uint8_t* out, float* scale, int t,
                                             float rstd, int shift, float* slot)
{
    const int nvec = p.hidden / kVec;
    constexpr float kNone = -100000.0f;
    float most = kNone, f[8], w[8];
#pragma unroll 1
    for (int i = t; i < nvec; i += TPR) {
        unpack8<F16>(load16<false>(s + i * kVec), f);
        load_weight(p, i, true, w);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (f[k] != 0.0f && w[k] != 0.0f)
                most = fmaxf(most, (float)(__builtin_amdgcn_frexp_expf(f[k]) + __builtin_amdgcn_frexp_expf(w[k])));
    }
    most = row_max<TPR>(most, slot);
    const int e = most == kNone ? 0 : (int)most;
    float top = 0.0f;
#pragma unroll 1
    for (int i = t; i < nvec; i += TPR) {
        unpack8<F16>(load16<false>(s + i * kVec), f);
        load_weight(p, i, true, w);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            top = fmaxf(top, fabsf(product(f[k], w[k], e)));
    }
    top = row_max<TPR>(top, slot);
    const float by = top > 0.0f ? kFp8Max / top : kFp8Max;
    if (t == 0)
        *scale = __builtin_amdgcn_ldexpf(__builtin_amdgcn_frexp_mantf(rstd) / by,
                                         __builtin_amdgcn_frexp_expf(rstd) + e - shift);
#pragma unroll 1
    for (int i = t; i < nvec; i += TPR) {
        unpack8<F16>(load16<false>(s + i * kVec), f);
        load_weight(p, i, true, w);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            f[k] = product(f[k], w[k], e) * by;
        *reinterpret_cast<uint64_t*>(out + i * kVec) = fp8x8(f);
    }
}

template <int TPR, int VPT, bool F16, bool RES, bool FP8>
__global__ __launch_bounds__(kThreads)
void rms_norm_kernel(const RmsParams p)
{
    constexpr int RPW = kThreads / TPR;
    __shared__ __attribute__((aligned(16))) float slot[RPW == 1 ? 20 : 4];
    const int t = threadIdx.x % TPR;
    const int nvec = p.hidden / kVec;
    const int64_t r = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
    if (RPW > 1 && r >= p.rows)
        return;
    const int64_t row = r * p.hidden;
    u32x4 x[VPT], res[RES ? VPT : 1];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int i = u * TPR + t;
        x[u] = u32x4{0, 0, 0, 0};
        if constexpr (RES)
            res[u] = u32x4{0, 0, 0, 0};
        if (i < nvec) {
            x[u] = load16<true>(p.x + row + i * kVec);
            if constexpr (RES)
                res[u] = load16<true>(p.residual + row + i * kVec);
        }
    }
    if constexpr (RES) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = u * TPR + t;
            float a[8], b[8];
            unpack8<F16>(x[u], a);
            unpack8<F16>(res[u], b);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                a[k] += b[k];
            x[u] = pack8<F16>(a);
            if (i < nvec)
                store16<true>(p.sum + row + i * kVec, x[u]);
        }
    }
    float ss, top;
    row_norm<TPR, VPT, F16, FP8, false>(x, p, t, nvec, 0, slot, ss, top);
    int shift = 0;
    float rstd = ss / (float)p.hidden + p.eps;
    // the same branch in every thread of the row
    if (__builtin_expect(rstd <= kMax && (ss >= kTinySum || p.eps >= kTinySum) &&
                             (!FP8 || (top >= kTinySum && top <= kMax)), 1)) {
        rstd = __builtin_amdgcn_rsqf(rstd);
    } else if (const float most = row_largest<TPR, VPT, F16>(x, slot + (RPW == 1 ? 16 : 0)); most == 0.0f) {
        rstd = rsqrt_full_range(ss / (float)p.hidden + p.eps);        // nothing but zeros, or NaN
    } else {
        shift = __builtin_amdgcn_frexp_expf(most);
        row_norm<TPR, VPT, F16, FP8, true>(x, p, t, nvec, shift, slot + (RPW == 1 ? 8 : 0), ss, top);
        const float eps = __builtin_amdgcn_ldexpf(p.eps, -2 * shift);
        // eps may be above x^2 by more than 2^128
        rstd = eps <= kMax ? rsqrt_full_range(ss / (float)p.hidden + eps)
                           : __builtin_amdgcn_ldexpf(rsqrt_full_range(p.eps), shift);
        if constexpr (FP8) {
            if (top < kTinySum && rstd > 0.0f) {
                small_to_8_bits<TPR, F16>(p, (RES ? p.sum : p.x) + row, static_cast<uint8_t*>(p.out) + row,
                                          p.scales + r, t, rstd, shift, slot + (RPW == 1 ? 16 : 0));
                return;
            }
        }
    }
    float f = 0.0f;
    if constexpr (FP8) {
        f = top > 0.0f ? kFp8Max / top : kFp8Max;
        if (t == 0)
            p.scales[r] = rstd > 0.0f ? rstd / f : NAN;       // 0: an infinity, whose products may all be NaN
    }
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int i = u * TPR + t;
        if (i < nvec) {
            float e[8], w[8], o[8];
            unpack8<F16>(x[u], e);
            load_weight(p, i, true, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float a = shift ? scaled(e[k], shift) : e[k];
                o[k] = FP8 ? a * w[k] * f : a * rstd * w[k];
            }
            if constexpr (FP8)
                *reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(p.out) + row + i * kVec) = fp8x8(o);
            else
                store16<true>(static_cast<uint16_t*>(p.out) + row + i * kVec, pack8<F16>(o));
        }
    }
}

// ---------------------------------------------------------------- backward

// What dx and dweight take of a row, of s * 2^-shift: rstd is 1 / sqrt(avg(s^2)
// + eps) of the scaled row, rstd_x of s itself, gn = sum g s (scaled).  shift is
// 0 unless the plain sums leave fp32's range.
struct RowStats {
    float rstd, rstd_x, gn;
    int shift;
};

template <int TPR, int VPT, bool F16, bool SCALED>
__device__ __forceinline__ void grad_sums(const u32x4 (&x)[VPT], const u32x4 (&dy)[VPT],
                                          const float (&w)[VPT][8], int shift, float* slot, float (&v)[2])
{
    v[0] = v[1] = 0.0f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        float f[8], d[8];
        unpack8<F16>(x[u], f);
        unpack8<F16>(dy[u], d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float e = SCALED ? scaled(f[k], shift) : f[k];
            v[0] = __builtin_fmaf(e, e, v[0]);
            v[1] = __builtin_fmaf(d[k] * w[u][k], e, v[1]);
        }
    }
    row_sums<TPR>(v, slot);
    forget_unpacked(x);
    forget_unpacked(dy);
}

// `slot`: 20 floats of LDS (of workgroups that hold one row), the first 8 of
// which the next row must not use.
template <int TPR, int VPT, bool F16>
__device__ __forceinline__ RowStats row_stats(const u32x4 (&x)[VPT], const u32x4 (&dy)[VPT],
                                              const float (&w)[VPT][8], int hidden, float eps, float* slot,
                                              float* spare)
{
    float v[2];
    grad_sums<TPR, VPT, F16, false>(x, dy, w, 0, slot, v);
    RowStats s;
    s.shift = 0;
    s.gn = v[1];
    s.rstd = v[0] / (float)hidden + eps;
    // sum g s may leave the range where its factors do not
    if (__builtin_expect(s.rstd <= kMax && (v[0] >= kTinySum || eps >= kTinySum) && fabsf(s.gn) <= kMax, 1)) {
        s.rstd = s.rstd_x = __builtin_amdgcn_rsqf(s.rstd);
        return s;
    }
    s.shift = __builtin_amdgcn_frexp_expf(row_largest<TPR, VPT, F16>(x, spare));
    grad_sums<TPR, VPT, F16, true>(x, dy, w, s.shift, spare + 4, v);
    s.gn = v[1];
    const float eps_s = __builtin_amdgcn_ldexpf(eps, -2 * s.shift);
    if (eps_s <= kMax) {
        s.rstd = rsqrt_full_range(v[0] / (float)hidden + eps_s);
        s.rstd_x = __builtin_amdgcn_ldexpf(s.rstd, -s.shift);
    } else {                     // avg(s^2) is below eps by more than 2^128
        s.rstd_x = rsqrt_full_range(eps);
        s.rstd = __builtin_amdgcn_ldexpf(s.rstd_x, s.shift);
    }
    return s;
}

// A workgroup's rows: TPR == 64 takes 4 at a time, one a wave.
template <int TPR, int VPT, bool F16, bool RES>
__global__ __launch_bounds__(kThreads, 2)
void rms_norm_backward_kernel(const RmsParams p)
{
    constexpr int RPW = kThreads / TPR;
    // two rows' sums in turn (the next row's may be written while this one's are
    // read: there is one barrier a row), then 12 for rows that are scaled
    __shared__ __attribute__((aligned(16))) float slot[RPW == 1 ? 28 : 4];
    extern __shared__ float joined[];       // RPW > 1: [3][hidden]
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int nvec = p.hidden / kVec;
    const int64_t first = (int64_t)blockIdx.x * p.rows_per_chunk;
    const int64_t end = first + p.rows_per_chunk < p.rows ? first + p.rows_per_chunk : p.rows;

    float w[VPT][8], dw[VPT][8];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        load_weight(p, u * TPR + t, u * TPR + t < nvec, w[u]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            dw[u][k] = 0.0f;
    }

    u32x4 x[VPT], dy[VPT], ds[RES ? VPT : 1], nx[VPT], ndy[VPT], nds[RES ? VPT : 1];
    const auto fetch = [&](int64_t r) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = u * TPR + t;
            nx[u] = ndy[u] = u32x4{0, 0, 0, 0};
            if (r < end && i < nvec) {
                nx[u] = load16<true>(p.x + r * p.hidden + i * kVec);
                ndy[u] = load16<true>(p.dy + r * p.hidden + i * kVec);
                if constexpr (RES)
                    nds[u] = load16<true>(p.residual + r * p.hidden + i * kVec);
            }
        }
    };
    fetch(first + sub);
    float* turn = slot;
    for (int64_t r = first + sub; r < end; r += RPW) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            x[u] = nx[u];
            dy[u] = ndy[u];
            if constexpr (RES)
                ds[u] = nds[u];
        }
        fetch(r + RPW);
        const RowStats s = row_stats<TPR, VPT, F16>(x, dy, w, p.hidden, p.eps, turn,
                                                    slot + (RPW == 1 ? 16 : 0));
        if constexpr (RPW == 1)
            turn = turn == slot ? slot + 8 : slot;
        const float c = s.gn * s.rstd / (float)p.hidden;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
                float f[8], d[8], a[8], o[8];
                unpack8<F16>(x[u], f);
                unpack8<F16>(dy[u], d);
                if constexpr (RES)
                    unpack8<F16>(ds[u], a);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float n = (s.shift ? scaled(f[k], s.shift) : f[k]) * s.rstd;
                    const float g = __builtin_fmaf(-n, c, d[k] * w[u][k]);
                    o[k] = RES ? __builtin_fmaf(g, s.rstd_x, a[k]) : g * s.rstd_x;
                    dw[u][k] = __builtin_fmaf(d[k], n, dw[u][k]);
                }
                store16<true>(static_cast<uint16_t*>(p.out) + r * p.hidden + i * kVec, pack8<F16>(o));
            }
        }
    }

    if (!p.dweight)
        return;
    if constexpr (RPW > 1) {            // the four waves' sums, in wave order
        if (sub > 0) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int i = u * TPR + t;
                if (i < nvec) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        joined[(sub - 1) * p.hidden + i * kVec + k] = dw[u][k];
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
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dw[u][k] += joined[j * p.hidden + i * kVec + k];
                }
            }
        }
    }
    float* to = p.chunks > 1 ? p.parts + (int64_t)blockIdx.x * p.hidden : p.dweight;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int i = u * TPR + t;
        if (i < nvec) {
            f32x4* a = reinterpret_cast<f32x4*>(to + i * kVec);
            a[0] = f32x4{dw[u][0], dw[u][1], dw[u][2], dw[u][3]};
            a[1] = f32x4{dw[u][4], dw[u][5], dw[u][6], dw[u][7]};
        }
    }
}

// dweight: the sums of the workgroups' parts.  8 threads side by side hold 4
// columns each, 32 such rows take every 32nd part.
__global__ __launch_bounds__(kThreads)
void rms_norm_parts_kernel(const RmsParams p)
{
    __shared__ f32x4 sums[32][8];
    const int col = (int)blockIdx.x * 32 + threadIdx.x % 8 * 4, row = threadIdx.x / 8;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < p.hidden) {
#pragma unroll 8
        for (uint32_t i = row; i < p.chunks; i += 32)
            s += *reinterpret_cast<const f32x4*>(p.parts + (int64_t)i * p.hidden + col);
    }
    sums[row][threadIdx.x % 8] = s;
    __syncthreads();
    if (row == 0 && col < p.hidden) {
#pragma unroll
        for (int i = 1; i < 32; ++i)
            s += sums[i][threadIdx.x];
        *reinterpret_cast<f32x4*>(p.dweight + col) = s;
    }
}

// ---------------------------------------------------------------- launches

// One wave a row up to this width, the whole workgroup above it.
constexpr int kWaveHidden = 1024;

using Fn = void (*)(RmsParams);

template <int TPR, int VPT>
Fn select(bool f16, bool res, bool fp8)
{
    if (f16)
        return res ? (fp8 ? rms_norm_kernel<TPR, VPT, true, true, true> : rms_norm_kernel<TPR, VPT, true, true, false>)
                   : (fp8 ? rms_norm_kernel<TPR, VPT, true, false, true> : rms_norm_kernel<TPR, VPT, true, false, false>);
    return res ? (fp8 ? rms_norm_kernel<TPR, VPT, false, true, true> : rms_norm_kernel<TPR, VPT, false, true, false>)
               : (fp8 ? rms_norm_kernel<TPR, VPT, false, false, true> : rms_norm_kernel<TPR, VPT, false, false, false>);
}

// Vectors a thread holds of a row.
int vectors_of(int hidden)
{
    const int nvec = hidden / kVec, threads = hidden <= kWaveHidden ? kWave : kThreads;
    return (nvec + threads - 1) / threads;
}

Fn select_forward(int hidden, bool f16, bool res, bool fp8)
{
    const int v = vectors_of(hidden);
    if (hidden <= kWaveHidden)
        return v == 1 ? select<64, 1>(f16, res, fp8) : select<64, 2>(f16, res, fp8);
    switch (v) {
    case 1: return select<256, 1>(f16, res, fp8);
    case 2: return select<256, 2>(f16, res, fp8);
    case 3: return select<256, 3>(f16, res, fp8);
    default: return select<256, 4>(f16, res, fp8);
    }
}

template <int TPR, int VPT>
Fn select_grad(bool f16, bool res)
{
    if (f16)
        return res ? rms_norm_backward_kernel<TPR, VPT, true, true> : rms_norm_backward_kernel<TPR, VPT, true, false>;
    return res ? rms_norm_backward_kernel<TPR, VPT, false, true> : rms_norm_backward_kernel<TPR, VPT, false, false>;
}

Fn select_backward(int hidden, bool f16, bool res)
{
    const int v = vectors_of(hidden);
    if (hidden <= kWaveHidden)
        return v == 1 ? select_grad<64, 1>(f16, res) : select_grad<64, 2>(f16, res);
    switch (v) {
    case 1: return select_grad<256, 1>(f16, res);
    case 2: return select_grad<256, 2>(f16, res);
    case 3: return select_grad<256, 3>(f16, res);
    default: return select_grad<256, 4>(f16, res);
    }
}

// Rows of a workgroup and workgroups of the backward pass.
struct Cut {
    int64_t chunks, each;
};

Cut cut_of(int64_t rows, int hidden)
{
    const int64_t at_once = hidden <= kWaveHidden ? 4 : 1;
    const int64_t most = (rows + at_once - 1) / at_once;
    const int64_t target = 256 * (vectors_of(hidden) == 1 ? 4 : 2);
    const int64_t chunks = target < most ? target : most;
    Cut c;
    c.each = ((rows + chunks - 1) / chunks + at_once - 1) / at_once * at_once;
    c.chunks = (rows + c.each - 1) / c.each;
    return c;
}

int check_sizes(int64_t rows, int32_t hidden)
{
    if (hidden < kVec || hidden > DIT_RMS_MAX_HIDDEN || hidden % kVec)
        return QKR_ERR_UNSUPPORTED;
    return rows < 0 || rows >= QKR_MAX_TOKENS ? QKR_ERR_SHAPE : QKR_OK;
}

int check(int64_t rows, int32_t hidden, int32_t dtype, int32_t param_dtype, float eps)
{
    if (dtype < QKR_BF16 || dtype > QKR_FP32 || param_dtype < QKR_BF16 || param_dtype > QKR_FP32)
        return QKR_ERR_ARG;
    if (dtype == QKR_FP32)
        return QKR_ERR_UNSUPPORTED;
    if (!(eps > 0.0f && isfinite(eps)))
        return QKR_ERR_ARG;
    return check_sizes(rows, hidden);
}

struct Buffer {
    const void* at;
    uint64_t bytes;
};

// Whether output `o` shares memory with `b` otherwise than by being `b` itself
// where that is allowed.
bool clash(const Buffer& o, const Buffer& b, bool same_allowed)
{
    return !(same_allowed && o.at == b.at) && overlaps(o.at, o.bytes, b.at, b.bytes);
}

hipError_t launch(Fn fn, int64_t blocks, size_t lds, RmsParams& p, void* stream)
{
    void* args[] = {&p};
    return hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)blocks), dim3(kThreads),
                           args, lds, static_cast<hipStream_t>(stream));
}

uint64_t param_bytes(const void* weight, int32_t hidden, int32_t param_dtype)
{
    return weight ? (uint64_t)hidden * (param_dtype == QKR_FP32 ? 4u : 2u) : 0;
}

}  // namespace

extern "C" int dit_rms_norm(const void* x, const void* residual, void* sum, void* y, float* scales,
                            int64_t rows, int32_t hidden, const void* weight, int32_t param_dtype,
                            float eps, int32_t dtype, void* stream)
{
    const int rc = check(rows, hidden, dtype, param_dtype, eps);
    if (rc != QKR_OK || rows == 0)
        return rc;
    if (!x || !y || !residual != !sum)
        return QKR_ERR_NULL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(sum) || !aligned16(y) || !aligned16(weight) ||
        (reinterpret_cast<uintptr_t>(scales) & 3u))
        return QKR_ERR_ALIGN;
    const uint64_t n = (uint64_t)rows * (uint64_t)hidden;
    const Buffer bx = {x, 2 * n}, br = {residual, residual ? 2 * n : 0}, bs = {sum, sum ? 2 * n : 0},
                 by = {y, scales ? n : 2 * n}, bc = {scales, scales ? (uint64_t)rows * 4 : 0},
                 bw = {weight, param_bytes(weight, hidden, param_dtype)};
    if (clash(bs, bx, true) || clash(bs, br, true) || clash(by, bx, !scales) || clash(by, br, !scales) ||
        clash(by, bs, false) || clash(bw, by, false) || clash(bw, bs, false) || clash(bc, bx, false) ||
        clash(bc, br, false) || clash(bc, bs, false) || clash(bc, by, false) || clash(bc, bw, false))
        return QKR_ERR_ARG;
    RmsParams p = {};
    p.x = static_cast<const uint16_t*>(x);
    p.residual = static_cast<const uint16_t*>(residual);
    p.sum = static_cast<uint16_t*>(sum);
    p.out = y;
    p.scales = scales;
    p.weight = weight;
    p.param_dtype = param_dtype;
    p.rows = rows;
    p.hidden = hidden;
    p.eps = eps;
    const int64_t blocks = hidden <= kWaveHidden ? (rows + 3) / 4 : rows;
    Fn fn = select_forward(hidden, dtype == QKR_FP16, residual != nullptr, scales != nullptr);
    return launch(fn, blocks, 0, p, stream) == hipSuccess ? QKR_OK : QKR_ERR_HIP;
}

extern "C" int64_t dit_rms_norm_backward_workspace_size(int64_t rows, int32_t hidden)
{
    const int rc = check_sizes(rows, hidden);
    if (rc != QKR_OK || rows == 0)
        return rc;
    const int64_t chunks = cut_of(rows, hidden).chunks;
    return chunks == 1 ? 0 : chunks * hidden * 4;
}

extern "C" int dit_rms_norm_backward(const void* dy, const void* s, const void* dsum, void* dx,
                                     int64_t rows, int32_t hidden, const void* weight,
                                     int32_t param_dtype, float* dweight, float eps, int32_t dtype,
                                     void* workspace, int64_t workspace_bytes, void* stream)
{
    const int rc = check(rows, hidden, dtype, param_dtype, eps);
    if (rc != QKR_OK || rows == 0)
        return rc;
    if (!dy || !s || !dx)
        return QKR_ERR_NULL;
    if (!aligned16(dy) || !aligned16(s) || !aligned16(dsum) || !aligned16(dx) || !aligned16(weight) ||
        !aligned16(dweight))
        return QKR_ERR_ALIGN;
    const int64_t need = dweight ? dit_rms_norm_backward_workspace_size(rows, hidden) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return QKR_ERR_WORKSPACE;
    if (need && !aligned16(workspace))
        return QKR_ERR_ALIGN;
    const uint64_t n = (uint64_t)rows * (uint64_t)hidden;
    const Buffer in[] = {{dy, 2 * n}, {dsum, dsum ? 2 * n : 0}, {s, 2 * n},
                         {weight, param_bytes(weight, hidden, param_dtype)}};
    const Buffer out[] = {{dx, 2 * n}, {dweight, dweight ? (uint64_t)hidden * 4 : 0},
                          {workspace, (uint64_t)need}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 4; ++j)
            if (clash(out[i], in[j], i == 0 && j < 2))
                return QKR_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (clash(out[i], out[j], false))
                return QKR_ERR_ARG;
    }
    RmsParams p = {};
    p.x = static_cast<const uint16_t*>(s);
    p.residual = static_cast<const uint16_t*>(dsum);
    p.dy = static_cast<const uint16_t*>(dy);
    p.out = dx;
    p.weight = weight;
    p.param_dtype = param_dtype;
    p.dweight = dweight;
    p.parts = static_cast<float*>(workspace);
    p.rows = rows;
    p.hidden = hidden;
    p.eps = eps;
    const Cut cut = cut_of(rows, hidden);
    p.chunks = (uint32_t)cut.chunks;
    p.rows_per_chunk = (uint32_t)cut.each;
    const size_t lds = dweight && hidden <= kWaveHidden ? (size_t)3 * hidden * 4 : 0;
    hipError_t err = launch(select_backward(hidden, dtype == QKR_FP16, dsum != nullptr), cut.chunks, lds, p, stream);
    if (err == hipSuccess && dweight && cut.chunks > 1)
        err = launch(rms_norm_parts_kernel, (hidden + 31) / 32, 0, p, stream);
    return err == hipSuccess ? QKR_OK : QKR_ERR_HIP;
}
