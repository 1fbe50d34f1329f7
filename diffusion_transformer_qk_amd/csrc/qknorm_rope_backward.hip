// qknorm_rope_backward.hip -- backward pass of the fused QK-norm + RoPE for
// gfx950 (see qknorm_rope_backward.h).
//
// Memory-bound: reads x and do once, writes dx once.  As in the forward pass a
// head is D / 8 lanes of 8 elements and a wave owns all heads of one tensor
// (Q or K) of a token; here it walks a run of tokens, so that its sums of
// dgamma stay in registers, 8 a lane.  With t = sum_d g x,
//   dx = r g - x r^3 t / D,
// so both sums of a head (x^2 and g x) are taken in one round of lane moves.
// The waves' sums are joined in the workgroup, written to the workspace and
// added in order by a second kernel: no atomics.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "qknorm_rope_backward.h"

namespace {

using namespace qkr_dev;
using qkr_host::aligned16;
using qkr_host::overlaps;

constexpr int kInterleaved = QKR_ROPE_INTERLEAVED;
constexpr int kThreads = 256;
constexpr int kWaves = 4;

struct BackParams {
    const uint16_t* x[2];      // element (t, h, d) of tensor s at x[s] + t*row_stride + h*D + d
    const uint16_t* grad[2];
    uint16_t* out[2];
    const float* gamma[2];
    float* dgamma[2];
    const void* cos;
    const void* sin;
    float* parts;              // [blocks][n_tensors][D]
    int64_t row_stride;
    int64_t tokens;
    int32_t heads;
    int32_t n_tensors;
    int32_t blocks;
    float eps;
};

__device__ __forceinline__ float lane_xor16(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F));
}

// Sum over the L lanes of a head; every lane ends with the same bits.
template <int L>
__device__ __forceinline__ float head_sum(float v)
{
    v += dpp<0xB1>(v);       // quad_perm [1,0,3,2]
    v += dpp<0x4E>(v);       // quad_perm [2,3,0,1]
    v += dpp<0x141>(v);      // row_half_mirror
    if constexpr (L >= 16)
        v += dpp<0x140>(v);  // row_mirror
    if constexpr (L == 32)
        v += lane_xor16(v);
    return v;
}

template <int L>
__device__ __forceinline__ float head_max(float v)
{
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x141>(v));
    if constexpr (L >= 16)
        v = fmaxf(v, dpp<0x140>(v));
    if constexpr (L == 32)
        v = fmaxf(v, lane_xor16(v));
    return v;
}

// The value of the lane whose dimensions are D / 2 away.
template <int L>
__device__ __forceinline__ float half_head_partner(float v)
{
    if constexpr (L == 32)
        return lane_xor16(v);
    else if constexpr (L == 16)
        return dpp_in_row<0x128>(v);
    else
        return __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x101F));
}

template <bool BF16_TABLE>
__device__ __forceinline__ void load_table8(const void* table, int64_t index, float f[8])
{
    if constexpr (BF16_TABLE)
        unpack8<false>(load16<false>(static_cast<const uint16_t*>(table) + index), f);
    else
        load_f32x8(static_cast<const float*>(table) + index, f);
}

// dn[d] = do[d] c[d] + do[partner] s[d], s[d] being the partner's sine with the
// sign of d's place in the pair.
template <int D, int STYLE, bool COS_BF16>
__device__ __forceinline__ void load_rotation(const BackParams& p, int64_t row, int d0, float c[8],
                                              float s[8])
{
    load_table8<COS_BF16>(p.cos, row * D + d0, c);
    if constexpr (STYLE == kInterleaved) {
        float f[8];
        load_table8<COS_BF16>(p.sin, row * D + d0, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[i] = i % 2 == 0 ? f[i ^ 1] : -f[i ^ 1];
    } else {
        load_table8<COS_BF16>(p.sin, row * D + (d0 + D / 2) % D, s);
        if (d0 >= D / 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] = -s[i];
        }
    }
}

constexpr float kTinySum = 0x1p-100f;

// dx of one head's slice in this lane, and its share of dgamma added to acc.
template <int D, int STYLE, bool F16>
__device__ __forceinline__ u32x4 head_backward(u32x4 xv, u32x4 gv, const float c[8], const float s[8],
                                               const float gamma[8], float eps, float acc[8])
{
    constexpr int L = D / kVec;
    float x[8], d[8], dn[8], g[8], o[8];
    unpack8<F16>(xv, x);
    unpack8<F16>(gv, d);
    float ss = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float other = STYLE == kInterleaved ? d[i ^ 1] : half_head_partner<L>(d[i]);
        dn[i] = __builtin_fmaf(d[i], c[i], other * s[i]);
        g[i] = dn[i] * gamma[i];
        ss = __builtin_fmaf(x[i], x[i], ss);
        t = __builtin_fmaf(g[i], x[i], t);
    }
    ss = head_sum<L>(ss);
    t = head_sum<L>(t);
    const float q = __builtin_fmaf(ss, 1.0f / D, eps);
    float r = __builtin_amdgcn_rsqf(q), rx = r;        // u = x * rx, dx = r (..)
    if (__builtin_expect(!(q <= 0x1.fffffep127f && (ss >= kTinySum || eps >= kTinySum) &&
                           fabsf(t) <= 0x1.fffffep127f), 0)) {
        // a plain sum is out of range: the same on x * 2^-e, e the exponent of
        // the head's largest |x| (the same branch in all its lanes)
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = fmaxf(m, fabsf(x[i]));
        const int e = __builtin_amdgcn_frexp_expf(head_max<L>(m));
        const float eps_s = __builtin_amdgcn_ldexpf(eps, -2 * e);
        if (!(eps_s <= 0x1.fffffep127f)) {
            r = rx = rsqrt_full_range(eps);            // mean(x^2) is far below eps
        } else {
            ss = t = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = __builtin_amdgcn_ldexpf(x[i], -e);
                ss = __builtin_fmaf(x[i], x[i], ss);
                t = __builtin_fmaf(g[i], x[i], t);
            }
            t = head_sum<L>(t);
            rx = rsqrt_full_range(__builtin_fmaf(head_sum<L>(ss), 1.0f / D, eps_s));
            r = __builtin_amdgcn_ldexpf(rx, -e);
        }
    }
    const float mean = rx * t * (1.0f / D);            // of g u
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float u = x[i] * rx;
        acc[i] = __builtin_fmaf(dn[i], u, acc[i]);
        o[i] = r * __builtin_fmaf(-u, mean, g[i]);
    }
    return pack8<F16>(o);
}

// Head iterations (of 64 / (D / 8) heads) whose loads are in flight together.
constexpr int kFlight = 4;

template <int D, int STYLE, bool PER_HEAD, bool COS_BF16, bool F16>
__global__ __launch_bounds__(kThreads)
void qknorm_rope_backward_kernel(const BackParams p)
{
    constexpr int L = D / kVec, HPI = kWave / L, U = kFlight;
    __shared__ float joined[kWaves][D];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int two = p.n_tensors == 2 ? 1 : 0;
    const int s = wave & two;
    const int tokens_at_once = kWaves >> two;
    const int d0 = lane % L * kVec, hs = lane / L;
    const int H = p.heads;

    // a contiguous run of tokens for each workgroup
    const int64_t steps = (p.tokens + tokens_at_once - 1) / tokens_at_once;
    const int64_t block = logical_block<-1>(blockIdx.x, gridDim.x);
    const int64_t first = steps * block / p.blocks, last = steps * (block + 1) / p.blocks;

    float gamma[8], acc[8] = {};
    load_f32x8(p.gamma[s] + d0, gamma);
    for (int64_t step = first; step < last; ++step) {
        const int64_t t = step * tokens_at_once + (wave >> two);
        if (t >= p.tokens)
            break;
        const int64_t at = t * p.row_stride + d0;
        const uint16_t* xr = p.x[s] + at;
        const uint16_t* gr = p.grad[s] + at;
        uint16_t* outr = p.out[s] + at;
        float c[8], sn[8];
        if constexpr (!PER_HEAD)
            load_rotation<D, STYLE, COS_BF16>(p, t, d0, c, sn);
        for (int h0 = 0; h0 < H; h0 += U * HPI) {
            u32x4 xv[U], gv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * HPI + hs;
                xv[u] = gv[u] = u32x4{0, 0, 0, 0};
                if (h < H) {
                    xv[u] = load16<true>(xr + h * D);
                    gv[u] = load16<true>(gr + h * D);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * HPI + hs;
                if constexpr (PER_HEAD)
                    load_rotation<D, STYLE, COS_BF16>(p, t * H + (h < H ? h : 0), d0, c, sn);
                const u32x4 o = head_backward<D, STYLE, F16>(xv[u], gv[u], c, sn, gamma, p.eps, acc);
                if (h < H)
                    store16<true>(outr + h * D, o);
            }
        }
    }

    // the head slots of the wave, then the waves of the tensor, in order
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int w = L; w < kWave; w *= 2)
            acc[i] += __shfl_xor(acc[i], w);
        if (lane < L)
            joined[wave][d0 + i] = acc[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.n_tensors * D; i += kThreads) {
        const int tensor = i / D, d = i % D;
        float sum = joined[tensor][d];
        for (int w = tensor + p.n_tensors; w < kWaves; w += p.n_tensors)
            sum += joined[w][d];
        p.parts[(block * p.n_tensors + tensor) * D + d] = sum;
    }
}

// dgamma: the workgroups' sums.  4 threads side by side hold 4 columns each, 64
// such rows take every 64th part.
template <int D>
__global__ __launch_bounds__(kThreads)
void qknorm_rope_dgamma_kernel(const BackParams p)
{
    __shared__ f32x4 sums[kThreads / 4][4];
    const int col = blockIdx.x * 16 + threadIdx.x % 4 * 4, row = threadIdx.x / 4;
    const int cols = p.n_tensors * D;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = row; i < p.blocks; i += kThreads / 4)
        s += *reinterpret_cast<const f32x4*>(p.parts + (int64_t)i * cols + col);
    sums[row][threadIdx.x % 4] = s;
    __syncthreads();
    if (row < 4) {
        for (int i = row + 4; i < kThreads / 4; i += 4)
            s += sums[i][threadIdx.x % 4];
        sums[row][threadIdx.x % 4] = s;
    }
    __syncthreads();
    if (row == 0) {
        s = (sums[0][threadIdx.x] + sums[1][threadIdx.x]) + (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
        *reinterpret_cast<f32x4*>(p.dgamma[col / D] + col % D) = s;
    }
}

using Fn = void (*)(BackParams);

template <int D, int STYLE, bool PER_HEAD, bool COS_BF16>
Fn select_type(bool f16)
{
    return f16 ? qknorm_rope_backward_kernel<D, STYLE, PER_HEAD, COS_BF16, true>
               : qknorm_rope_backward_kernel<D, STYLE, PER_HEAD, COS_BF16, false>;
}

template <int D, int STYLE>
Fn select_table(bool per_head, bool cos_bf16, bool f16)
{
    if (per_head)
        return cos_bf16 ? select_type<D, STYLE, true, true>(f16) : select_type<D, STYLE, true, false>(f16);
    return cos_bf16 ? select_type<D, STYLE, false, true>(f16) : select_type<D, STYLE, false, false>(f16);
}

template <int D>
Fn select_style(int style, bool per_head, bool cos_bf16, bool f16)
{
    return style == kInterleaved ? select_table<D, QKR_ROPE_INTERLEAVED>(per_head, cos_bf16, f16)
                                 : select_table<D, QKR_ROPE_ROTATE_HALF>(per_head, cos_bf16, f16);
}

int check_sizes(int64_t tokens, int32_t head_dim)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return QKR_ERR_UNSUPPORTED;
    return tokens < 0 || tokens >= QKR_MAX_TOKENS ? QKR_ERR_SHAPE : QKR_OK;
}

// Workgroups of a call: enough to fill the chip, none without a token.
int64_t blocks_of(int64_t tokens)
{
    const int64_t steps = (tokens + 1) / 2;
    return steps < QKR_BACKWARD_MAX_BLOCKS ? steps : QKR_BACKWARD_MAX_BLOCKS;
}

}  // namespace

extern "C" int64_t qknorm_rope_backward_workspace_size(int64_t tokens, int32_t head_dim)
{
    const int rc = check_sizes(tokens, head_dim);
    return rc != QKR_OK ? rc : blocks_of(tokens) * 2 * head_dim * 4;
}

extern "C" int qknorm_rope_backward(const qkr_grad_tensor* qkv, const qkr_grad_tensor* q,
                                    const qkr_grad_tensor* k, int64_t tokens, int32_t heads,
                                    int32_t head_dim, const float* q_gamma, const float* k_gamma,
                                    float* dq_gamma, float* dk_gamma, float eps, const void* cos,
                                    const void* sin, int32_t cos_layout, int32_t cos_dtype,
                                    int32_t style, int32_t dtype, void* workspace,
                                    int64_t workspace_bytes, void* stream)
{
    if (dtype < QKR_BF16 || dtype > QKR_FP32 || cos_dtype < QKR_BF16 || cos_dtype > QKR_FP32 ||
        (cos_layout != QKR_COS_SHARED && cos_layout != QKR_COS_PER_HEAD) ||
        (style != QKR_ROPE_INTERLEAVED && style != QKR_ROPE_ROTATE_HALF) || !(eps > 0.0f) ||
        !isfinite(eps))
        return QKR_ERR_ARG;
    if (dtype == QKR_FP32 || cos_dtype == QKR_FP16)
        return QKR_ERR_UNSUPPORTED;
    int rc = check_sizes(tokens, head_dim);
    if (rc != QKR_OK)
        return rc;
    if (heads < 1 || heads > QKR_MAX_HEADS)
        return QKR_ERR_SHAPE;
    if ((qkv != nullptr) == (q != nullptr || k != nullptr))
        return QKR_ERR_MODE;
    const bool has_q = qkv || q, has_k = qkv || k;
    if ((has_q && (!q_gamma || !dq_gamma)) || (has_k && (!k_gamma || !dk_gamma)))
        return QKR_ERR_NULL;
    const qkr_grad_tensor* given[] = {qkv, q, k};
    if (tokens > 0) {
        for (const qkr_grad_tensor* t : given)
            if (t && (!t->grad || !t->x || !t->out))
                return QKR_ERR_NULL;
        if (!cos || !sin)
            return QKR_ERR_NULL;
    }
    const int64_t need = qknorm_rope_backward_workspace_size(tokens, head_dim);
    if (need && (!workspace || workspace_bytes < need))
        return QKR_ERR_WORKSPACE;
    for (const qkr_grad_tensor* t : given)
        if (t && (!aligned16(t->grad) || !aligned16(t->x) || !aligned16(t->out)))
            return QKR_ERR_ALIGN;
    const void* others[] = {q_gamma, k_gamma, dq_gamma, dk_gamma, cos, sin, workspace};
    for (const void* at : others)
        if (!aligned16(at))
            return QKR_ERR_ALIGN;

    const uint64_t row = (uint64_t)heads * head_dim * (qkv ? 3 : 1);
    const uint64_t bytes = (uint64_t)tokens * row * 2;
    const uint64_t g = (uint64_t)head_dim * 4;
    const uint64_t table = (uint64_t)tokens * (cos_layout == QKR_COS_PER_HEAD ? heads : 1) * head_dim *
                           (cos_dtype == QKR_FP32 ? 4 : 2);
    struct Range { const void* at; uint64_t n; } in[10], out[6];
    int n_in = 0, n_out = 0;
    for (const qkr_grad_tensor* t : given)
        if (t) {
            if (t->out != t->grad && overlaps(t->out, bytes, t->grad, bytes))
                return QKR_ERR_ARG;
            out[n_out++] = Range{t->out, bytes};
            in[n_in++] = Range{t->x, bytes};
        }
    if (q && k && (overlaps(q->out, bytes, k->grad, bytes) || overlaps(k->out, bytes, q->grad, bytes)))
        return QKR_ERR_ARG;
    const int n_data = n_out;
    if (has_q) {
        in[n_in++] = Range{q_gamma, g};
        out[n_out++] = Range{dq_gamma, g};
    }
    if (has_k) {
        in[n_in++] = Range{k_gamma, g};
        out[n_out++] = Range{dk_gamma, g};
    }
    in[n_in++] = Range{cos, table};
    in[n_in++] = Range{sin, table};
    out[n_out++] = Range{workspace, (uint64_t)need};
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlaps(out[i].at, out[i].n, in[j].at, in[j].n))
                return QKR_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].at, out[i].n, out[j].at, out[j].n))
                return QKR_ERR_ARG;
        for (const qkr_grad_tensor* t : given)
            if (t && i >= n_data && overlaps(out[i].at, out[i].n, t->grad, bytes))
                return QKR_ERR_ARG;
    }

    BackParams p = {};
    const int64_t hd = (int64_t)heads * head_dim;
    const auto add = [&](const qkr_grad_tensor* t, int64_t at, const float* gamma, float* dgamma) {
        const int i = p.n_tensors++;
        p.grad[i] = static_cast<const uint16_t*>(t->grad) + at;
        p.x[i] = static_cast<const uint16_t*>(t->x) + at;
        p.out[i] = static_cast<uint16_t*>(t->out) + at;
        p.gamma[i] = gamma;
        p.dgamma[i] = dgamma;
    };
    if (qkv) {
        add(qkv, 0, q_gamma, dq_gamma);
        add(qkv, hd, k_gamma, dk_gamma);
    } else {
        if (q)
            add(q, 0, q_gamma, dq_gamma);
        if (k)
            add(k, 0, k_gamma, dk_gamma);
    }
    p.cos = cos;
    p.sin = sin;
    p.parts = static_cast<float*>(workspace);
    p.row_stride = (int64_t)row;
    p.tokens = tokens;
    p.heads = heads;
    p.blocks = (int32_t)blocks_of(tokens);
    p.eps = eps;
    const bool per_head = cos_layout == QKR_COS_PER_HEAD, cos_bf16 = cos_dtype == QKR_BF16,
               f16 = dtype == QKR_FP16;
    Fn fn = head_dim == 64    ? select_style<64>(style, per_head, cos_bf16, f16)
            : head_dim == 128 ? select_style<128>(style, per_head, cos_bf16, f16)
                              : select_style<256>(style, per_head, cos_bf16, f16);
    Fn join = head_dim == 64    ? qknorm_rope_dgamma_kernel<64>
              : head_dim == 128 ? qknorm_rope_dgamma_kernel<128> : qknorm_rope_dgamma_kernel<256>;
    void* args[] = {&p};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t err = hipSuccess;
    if (p.blocks)
        err = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)p.blocks),
                              dim3(kThreads), args, 0, st);
    if (err == hipSuccess)
        err = hipLaunchKernel(reinterpret_cast<const void*>(join),
                              dim3((unsigned)(p.n_tensors * head_dim / 16)), dim3(kThreads), args, 0, st);
    return err == hipSuccess ? QKR_OK : QKR_ERR_HIP;
}
