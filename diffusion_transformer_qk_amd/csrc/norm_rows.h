// norm_rows.h -- what the norms over whole rows (layer norm, RMS norm) share:
// rows held by one wave or by the four waves of a workgroup, parameters of any
// type, sums over a row.  Internal header.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "device_common.h"
#include "qknorm_rope.h"

namespace qkr_rows {

using namespace qkr_dev;

constexpr int kThreads = 256;

// Sums of squares at or above this keep full fp32 precision.
constexpr float kTinySum = 0x1p-100f;

// 8 parameters from entry i of a [hidden] row of param_dtype at `at`.
__device__ __forceinline__ void load_params(const void* at, int64_t i, int32_t dtype, float f[8])
{
    if (dtype == QKR_FP32)
        load_f32x8(static_cast<const float*>(at) + i, f);
    else if (dtype == QKR_FP16)
        unpack8<true>(load16<false>(static_cast<const uint16_t*>(at) + i), f);
    else
        unpack8<false>(load16<false>(static_cast<const uint16_t*>(at) + i), f);
}

// Make the compiler forget what v holds, so that the fp32 values unpacked from
// it are unpacked again for each pass instead of being kept across them: for
// the longest rows, whose registers would not allow two workgroups a CU (kept,
// the values save a tenth of the backward pass's instructions).
template <int VPT>
__device__ __forceinline__ void forget_unpacked(const u32x4 (&v)[VPT])
{
    if constexpr (VPT == 4) {
#pragma unroll
        for (int u = 0; u < VPT; ++u)
            __asm__ volatile("" : "+v"(const_cast<u32x4&>(v[u])));
    }
}

// Sum over the wave by lane moves alone; every lane ends with the same bits.
__device__ __forceinline__ float wave_total(float v)
{
    v += dpp<0xB1>(v);      // quad_perm [1,0,3,2]
    v += dpp<0x4E>(v);      // quad_perm [2,3,0,1]
    v += dpp<0x141>(v);     // row_half_mirror
    v += dpp<0x140>(v);     // row_mirror: each 16-lane row's total in all its lanes
    const uint32_t a = __float_as_uint(v);
    const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    const uint32_t b = __float_as_uint(v);
    const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}

// Sums over the row's threads, the same bits in each.  `slot`: 4 floats of LDS
// per value, which may be used again after the workgroup's next barrier.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* slot)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = wave_total(v[i]);
    if constexpr (TPR > kWave) {
        if (threadIdx.x % kWave == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                slot[4 * i + threadIdx.x / kWave] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const f32x4 s = *reinterpret_cast<const f32x4*>(slot + 4 * i);
            v[i] = (s[0] + s[1]) + (s[2] + s[3]);
        }
    }
}

template <int TPR>
__device__ __forceinline__ float row_max(float v, float* slot)
{
    v = wave_max(v);
    if constexpr (TPR > kWave) {
        __syncthreads();
        if (threadIdx.x % kWave == 0)
            slot[threadIdx.x / kWave] = v;
        __syncthreads();
        v = fmaxf(fmaxf(slot[0], slot[1]), fmaxf(slot[2], slot[3]));
        __syncthreads();
    }
    return v;
}

}  // namespace qkr_rows
