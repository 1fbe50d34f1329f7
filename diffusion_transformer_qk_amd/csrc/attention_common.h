// attention_common.h -- tiles, matrix products and lane moves shared by the
// attention kernels (forward and backward).  Internal header.
//
// Fragments of v_mfma_f32_32x32x16 (lane = 32 g + n, g = 0 or 1):
//   A (32 x 16): lane holds row n, columns 8g .. 8g+7      (4 registers)
//   B (16 x 32): lane holds column n, rows 8g .. 8g+7      (4 registers)
//   C (32 x 32): lane holds column n, rows 8 (i/4) + 4g + i%4, i = 0..15
// A product over k may visit k in any order as long as A and B agree.  The C
// registers 8s .. 8s+7 of a tile, packed to 16 bits, are therefore a B operand
// as they stand: they hold k = 16s + 8 (j/4) + 4g + j%4 (j = 0..7), and the
// other operand is read from LDS in that order (tr_fragment below).
//
// A tile in LDS is rows of head_dim 16-bit elements, as they lie in memory,
// with the 16-byte chunks of each row permuted: chunk c of row r is stored at
// c ^ swizzle(r).  Rows are a multiple of 128 bytes apart, so without it the
// lanes of a fragment read, which go down the rows, would meet in the same
// banks.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "device_common.h"

namespace qkr_attn {

using namespace qkr_dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kRawBuffer = 0x00020000u;   // raw buffer resource, 32-bit data

template <bool F16>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const f32x2 pr = {a, b};
    if constexpr (F16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, f16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2));
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ uint32_t scalar(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// C registers 8s .. 8s+7 as the B operand of k step s.
template <bool F16>
__device__ __forceinline__ u32x4 pack_b(const f32x16& c, int s)
{
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = pack2<F16>(c[8 * s + 2 * j], c[8 * s + 2 * j + 1]);
    return w;
}

// The value of lane ^ 32 combined with the own one; both lanes get the same bits.
__device__ __forceinline__ float half_max(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float half_sum(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// swizzle(row): 16 rows map to 16 different chunks (8 for head_dim 64, where
// two rows share a line of the banks), and the 4 rows of a transposed read to
// 4 different groups of 4 chunks (2 of 4).
template <int D>
__device__ __forceinline__ int swizzle(int row)
{
    if constexpr (D == 64)
        return (((row >> 1) & 1) << 2) | (((row >> 2) & 1) << 1) | ((row >> 3) & 1);
    else
        return ((row & 3) << 2) | ((row >> 2) & 3);
}

// Rows of a tile are staged straight into LDS, 64 lanes x 16 bytes an
// instruction, in the order of LDS: the permutation is in the addresses that
// the lanes read.  Rows from `rows` on read as zero (the buffer's range ends
// there; this needs a row stride of at least head_dim).
template <int D, int ROWS, int NW>
struct Stager {
    static constexpr int kRowBytes = 2 * D;
    static constexpr int kRowsPer = 1024 / kRowBytes;              // rows of one instruction
    static constexpr int kPer = ROWS * kRowBytes / 1024 / NW;      // instructions of one wave
    static_assert(ROWS * kRowBytes % (1024 * NW) == 0, "whole instructions");
    uint32_t off[kPer];

    __device__ __forceinline__ void init(int wave, int lane, int64_t row_stride)
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int row = (wave * kPer + i) * kRowsPer + lane * 16 / kRowBytes;
            const int slot = (lane * 16 % kRowBytes) / 16;
            off[i] = (uint32_t)(row * (int)(row_stride * 2) + ((slot ^ swizzle<D>(row)) << 4));
        }
    }

    // `base`: the tile's first row; `lds`: byte address of the tile in LDS.
    __device__ __forceinline__ void load(const uint16_t* base, int64_t row_stride, int rows, uint32_t lds,
                                         int wave) const
    {
        const int n = rows < 0 ? 0 : rows > ROWS ? ROWS : rows;
        const int bytes = n ? (n - 1) * (int)(row_stride * 2) + kRowBytes : 0;
        const uint64_t a = reinterpret_cast<uint64_t>(base);
        const u32x4 rsrc = {scalar((uint32_t)a), scalar((uint32_t)(a >> 32) & 0xffffu),
                            scalar((uint32_t)bytes), kRawBuffer};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            dma16(rsrc, off[i], lds + (wave * kPer + i) * 1024, i == 0);
    }

    // 64 x 16 bytes from buffer offsets `off` to LDS at `lds` + lane * 16.
    // Written in assembly because the compiler, which cannot tell the halves
    // of a double buffer apart, would wait for these loads before the next
    // LDS read; wait_staged() waits for them.  The no-ops are the wait states
    // after a scalar register written by the vector unit (the first load of a
    // resource) and after m0.
    static __device__ __forceinline__ void dma16(u32x4 rsrc, uint32_t off, uint32_t lds, bool first)
    {
        const uint32_t at = scalar(lds);
        if (first)
            __asm__ volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                             : : "v"(off), "s"(rsrc), "s"(at) : "memory");
        else
            __asm__ volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                             : : "v"(off), "s"(rsrc), "s"(at) : "memory");
    }
};

// 64 x 4 bytes, the same way.
__device__ __forceinline__ void dma4(u32x4 rsrc, uint32_t off, uint32_t lds)
{
    __asm__ volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds"
                     : : "v"(off), "s"(rsrc), "s"(scalar(lds)) : "memory");
}

// Waits for this wave's staged tiles; after the barrier that follows, every
// wave's are there.
__device__ __forceinline__ void wait_staged()
{
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    return (uint32_t)reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) const void*)p);
}

// The A or B fragment of rows n (of a 32-row block) and columns 16 kk + 8g..:
// `at` is the byte offset of the lane's row start with (g ^ swizzle) applied.
template <int D>
__device__ __forceinline__ uint32_t row_offset(int lane)
{
    const int n = lane & 31, g = lane >> 5;
    return n * 2 * D + ((g ^ swizzle<D>(n)) << 4);
}

template <int D>
__device__ __forceinline__ u32x4 row_fragment(const char* tile, uint32_t at, int block, int kk)
{
    return *reinterpret_cast<const u32x4*>(tile + block * 64 * D + (at ^ (kk << 5)));
}

// The fragment whose lane index runs over 32 columns (column block db) and
// whose k runs over the rows of k step s of a 32-row block, in the order of
// packed C registers: two transposed reads, of rows 16s + 4g .. +3 and 8 more.
template <int D>
__device__ __forceinline__ uint32_t tr_offset(int lane)
{
    const int l = lane & 15, g = lane >> 5;
    const int row = 4 * g + (l >> 2);
    const int chunk = ((lane >> 4) & 1) * 2 + ((l & 3) >> 1);
    return row * 2 * D + ((chunk ^ swizzle<D>(row)) << 4) + (l & 1) * 8;
}

__device__ __forceinline__ u32x2 tr_read(const char* p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)const_cast<char*>(p)));
}

template <int D>
__device__ __forceinline__ u32x4 tr_fragment(const char* tile, uint32_t at, int block, int s, int db)
{
    constexpr int kFlip = D == 64 ? 16 : 32;      // swizzle(row + 8) ^ swizzle(row), in bytes
    const char* t = tile + block * 64 * D + s * 32 * D;
    const u32x2 a = tr_read(t + (at ^ (db << 6)));
    const u32x2 b = tr_read(t + 16 * D + (at ^ (db << 6) ^ kFlip));
    return u32x4{a[0], a[1], b[0], b[1]};
}

// Column n (this lane's) of a C block, times `f`, as 16-bit elements d0 + 0..31
// at `row`: the halves of the wave trade groups of 4 so that each lane stores
// 16 bytes at a time.
template <bool F16>
__device__ __forceinline__ void store_column(uint16_t* row, const f32x16& c, float f, int g, bool valid)
{
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t a = pack2<F16>(c[4 * i + 2 * j] * f, c[4 * i + 2 * j + 1] * f);
            const uint32_t b = pack2<F16>(c[4 * i + 4 + 2 * j] * f, c[4 * i + 4 + 2 * j + 1] * f);
            const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
            w[j] = r[0];
            w[2 + j] = r[1];
        }
        if (valid)
            store16<false>(row + 8 * (i + g), w);
    }
}

// The same in fp32.
__device__ __forceinline__ void store_column_f32(float* row, const f32x16& c, float f, int g, bool valid)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (valid)
            *reinterpret_cast<f32x4*>(row + 8 * i + 4 * g) =
                f32x4{c[4 * i] * f, c[4 * i + 1] * f, c[4 * i + 2] * f, c[4 * i + 3] * f};
}

}  // namespace qkr_attn
