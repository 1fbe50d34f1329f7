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
// A tile in LDS is laid out in blocks of 32 rows, a block in slabs of 32
// columns, a slab as its 32 rows of 64 bytes with the 16-byte chunks of row r
// permuted: chunk c is stored at c ^ ((r / 4) % 4).  So
//   * an A or B fragment of rows (32 rows, 16 columns: half a slab) touches
//     every bank evenly, and so does a transposed read (8 rows, one slab);
//   * a lane's address in a slab takes two values for either kind of read (the
//     half of the slab; the upper or lower 8 rows): all else is an immediate
//     offset, and four registers address a whole tile;
//   * 64 bytes of 16 rows are one load of a wave straight into LDS.
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
// Query rows a key head, of a sample or a packed sequence, up to which p and ds go
// into their products in two terms (dit_attention.h).
constexpr int kTwoTermRows = 32;
constexpr uint32_t kRawBuffer = 0x00020000u;   // raw buffer resource, 32-bit data

// The (pair, part) of hardware block `bid`, for `pairs` (sample, key head) pairs
// of `parts` blocks each.  The dispatcher deals consecutive blocks to
// consecutive dies, and the blocks of a pair read the same keys, so a pair
// stays on one die, with its L2: die d takes pairs d, d + 8, ...  (Neighbouring
// pairs, which are of one sample and so of one length, go to different dies.)
// The last pairs % 8 are cut into eighths, one a die.
//
// A die takes its pairs one after another, or (IN_TURN) each part of all of them
// before the next part.  Parts of very different work, as packed sequences make
// them, then do not leave a whole pair's longest for the end: forward over
// sequences of 4096, 1560, 1024, 777, 512 and 221, 40 heads of 128, 443 us one
// after another and 414 in turn (448 and 428 from the shortest to the longest); one
// sequence of 16384 4836 and 4866.  The backward pass, which reads four matrices,
// gains 2% there and loses 9% on the long one, and keeps to one after another.
template <bool IN_TURN = false>
struct BlockOf {
    uint32_t pair;
    int32_t part;

    __device__ __forceinline__ BlockOf(uint32_t bid, uint32_t pairs, uint32_t parts)
    {
        const uint32_t whole = pairs / kXcds * kXcds;
        const uint32_t die = bid % kXcds, local = bid / kXcds;
        if (bid < whole * parts) {
            const uint32_t mine = pairs / kXcds;
            pair = (IN_TURN ? local % mine : local / parts) * kXcds + die;
            part = IN_TURN ? local / mine : local % parts;
        } else {
            const uint32_t blocks = (pairs - whole) * parts;
            const uint32_t at = (uint32_t)logical_block<-1>(bid - whole * parts, blocks);
            pair = whole + at / parts;
            part = at % parts;
        }
    }
};

// Packed sequences: sequence i of `sequences` has rows offsets[i] .. offsets[i + 1]
// - 1 of a buffer of `total` rows.  The buffer's rows before the first and behind
// the last are counted as sequences 0 and sequences + 1 here (the others are one
// further), which have no keys.  Offsets are clamped to the buffer, so that none,
// whatever it holds, leads out of it.
struct Rows {
    const int32_t* offsets;
    int32_t sequences, total;

    __device__ __forceinline__ int first(int seq) const
    {
        if (seq == 0)
            return 0;
        if (seq > sequences + 1)
            return total;
        const int at = offsets[seq - 1];
        return at < 0 ? 0 : at > total ? total : at;
    }

    __device__ __forceinline__ bool rest(int seq) const { return seq == 0 || seq > sequences; }
};

// Rows are dealt to workgroups in blocks of SIZE rows (times `group`) of one
// sequence: sequence i has the blocks from first(i) * group / SIZE + i on, which
// leaves each as many as it can need, so that block numbers follow from the
// offsets without a sum over the sequences before.
template <int SIZE>
__device__ __forceinline__ int first_block(const Rows& r, int group, int seq)
{
    return r.first(seq) * group / SIZE + seq;
}

// The sequence of block `block`: 64 of them are looked at a time, by the lanes of
// a wave, which all get the answer.
template <int SIZE>
__device__ __forceinline__ int sequence_of(const Rows& r, int group, int block)
{
    const int lane = threadIdx.x % kWave;
    int low = 0, count = r.sequences + 2;
    while (count > 1) {
        const int step = (count + kWave - 1) / kWave, i = lane * step;
        const bool before = i < count && first_block<SIZE>(r, group, low + i) <= block;
        const int n = __builtin_popcountll(__ballot(before));      // a run from lane 0 on
        const int skip = n > 0 ? (n - 1) * step : 0;
        low += skip;
        count = count - skip < step ? count - skip : step;
    }
    return __builtin_amdgcn_readfirstlane(low);
}

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

// What the rounding of pack_b left: the difference, packed the same way.
template <bool F16>
__device__ __forceinline__ u32x4 pack_rest(const f32x16& c, int s, u32x4 packed)
{
    float f[8];
    unpack8<F16>(packed, f);
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = pack2<F16>(c[8 * s + 2 * j] - f[2 * j], c[8 * s + 2 * j + 1] - f[2 * j + 1]);
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

typedef __attribute__((address_space(3))) const u32x4* LdsVec;
typedef __attribute__((address_space(3))) const f32x4* LdsFloats;
typedef __attribute__((address_space(3))) s16x4* LdsQuad;

constexpr int kSlab = 2048;                        // 32 rows of 64 bytes

template <int D>
constexpr int block_bytes() { return 64 * D; }     // 32 rows

__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    return (uint32_t)reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) const void*)p);
}

// Byte addresses of this lane's part of a tile.
struct TileAt {
    uint32_t row[2];     // fragment of rows: half 0 and 1 of a slab
    uint32_t tr[2];      // transposed read: rows 0 and 8 of a k step

    __device__ __forceinline__ TileAt(uint32_t lds, int lane)
    {
        const int n = lane & 31, g = lane >> 5, l = lane & 15;
        row[0] = lds + n * 64 + ((g ^ ((n >> 2) & 3)) << 4);
        row[1] = lds + n * 64 + (((2 + g) ^ ((n >> 2) & 3)) << 4);
        const int r = 4 * g + (l >> 2), chunk = ((lane >> 4) & 1) * 2 + ((l & 3) >> 1);
        tr[0] = lds + r * 64 + ((chunk ^ g) << 4) + (l & 1) * 8;
        tr[1] = lds + (r + 8) * 64 + ((chunk ^ g ^ 2) << 4) + (l & 1) * 8;
    }

    // To the other half of a double buffer whose halves are `bytes` (a power
    // of two, to which the buffer is aligned) apart.
    __device__ __forceinline__ void flip(uint32_t bytes)
    {
        row[0] ^= bytes;
        row[1] ^= bytes;
        tr[0] ^= bytes;
        tr[1] ^= bytes;
    }
};

// The A or B fragment of 32 rows and columns 16 kk .. 16 kk + 15; `off`: the
// block's offset from the tile address.
__device__ __forceinline__ u32x4 row_fragment(const TileAt& at, int off, int kk)
{
    return *reinterpret_cast<LdsVec>(at.row[kk & 1] + (off + (kk >> 1) * kSlab));
}

// The fragment whose lane index runs over the 32 columns of slab c and whose k
// runs over rows 16s .. 16s + 15 of the block, in the order of packed C
// registers: two transposed reads of 8 rows.
__device__ __forceinline__ u32x4 tr_fragment(const TileAt& at, int off, int s, int c)
{
    const int o = off + c * kSlab + s * 1024;
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<LdsQuad>(at.tr[0] + o)));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<LdsQuad>(at.tr[1] + o)));
    return u32x4{a[0], a[1], b[0], b[1]};
}

// Rows of a tile are staged straight into LDS in groups of 16 rows; a wave
// stages one group (all slabs) or several.  Rows from `rows` on read as zero:
// the buffer's range ends there (this needs a row stride of at least head_dim).
template <int D>
struct Stager {
    uint32_t off;

    __device__ __forceinline__ Stager(int lane, int64_t row_stride)
        : off((uint32_t)((lane >> 2) * (int)(row_stride * 2) + (((lane & 3) ^ ((lane >> 4) & 3)) << 4)))
    {
    }

    // Group `group` of the tile whose first row is at `base` and which starts
    // at `lds`; base, row_stride, rows, lds and group are the wave's.
    __device__ __forceinline__ void load(const uint16_t* base, int64_t row_stride, int rows, uint32_t lds,
                                         int group) const
    {
        const int left = rows - 16 * group;
        const int n = left < 0 ? 0 : left > 16 ? 16 : left;
        const int bytes = n ? (n - 1) * (int)(row_stride * 2) + 2 * D : 0;
        const uint64_t a = reinterpret_cast<uint64_t>(base + 16 * group * row_stride);
        const u32x4 rsrc = {scalar((uint32_t)a), scalar((uint32_t)(a >> 32) & 0xffffu),
                            scalar((uint32_t)bytes), kRawBuffer};
        const uint32_t to = lds + (group >> 1) * block_bytes<D>() + (group & 1) * 1024;
        dma_row_group(rsrc, off, to);
    }

    // 64 x 16 bytes of each slab c, from buffer offsets off + 64 c to LDS at `to` +
    // c * kSlab + lane * 16 (the instruction's offset counts in both, so m0 moves
    // by the rest).  Written in assembly because the compiler, which cannot tell
    // the halves of a double buffer apart, would wait for these loads before the
    // next LDS read; wait_staged() waits for them.  The no-ops are the wait states
    // after a scalar register written by the vector unit (a resource just formed,
    // or fetched back from a lane in which the compiler kept it) and after m0.
    // All slabs are one block of assembly: between two, the compiler might fetch
    // a part of the resource back and would not know what the next one waits for.
    static __device__ __forceinline__ void dma_row_group(u32x4 rsrc, uint32_t off, uint32_t to)
    {
#define QKR_FIRST_SLAB "s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
#define QKR_NEXT_SLAB(offset) \
    "\n\ts_add_u32 m0, m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen offset:" #offset " lds"
#define QKR_SLABS(text) \
    __asm__ volatile(text : : "v"(off), "s"(rsrc), "s"(scalar(to)), "i"(kSlab - 64) : "memory", "scc")
        if constexpr (D == 64)
            QKR_SLABS(QKR_FIRST_SLAB QKR_NEXT_SLAB(64));
        else if constexpr (D == 128)
            QKR_SLABS(QKR_FIRST_SLAB QKR_NEXT_SLAB(64) QKR_NEXT_SLAB(128) QKR_NEXT_SLAB(192));
        else
            QKR_SLABS(QKR_FIRST_SLAB QKR_NEXT_SLAB(64) QKR_NEXT_SLAB(128) QKR_NEXT_SLAB(192)
                      QKR_NEXT_SLAB(256) QKR_NEXT_SLAB(320) QKR_NEXT_SLAB(384) QKR_NEXT_SLAB(448));
#undef QKR_SLABS
#undef QKR_NEXT_SLAB
#undef QKR_FIRST_SLAB
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

// Keeps a fragment in registers from here on: without it the compiler, which
// does not know that the loads above count as well, waits for fragments loaded
// ahead of a loop again in each of its rounds.
__device__ __forceinline__ void settle(u32x4& f) { __asm__ volatile("" : "+v"(f)); }

// In a branch that few tiles take: keeps the compiler from turning it into
// selects that all of them execute.
__device__ __forceinline__ void keep_branch() { __asm__ volatile("" ::: "memory"); }

// Column n (this lane's) of a C block, times `f` (zeros unless `keep`), as
// 16-bit elements d0 + 0..31 at `row`: the halves of the wave trade groups of 4
// so that each lane stores 16 bytes at a time.
template <bool F16>
__device__ __forceinline__ void store_column(uint16_t* row, const f32x16& c, float f, int g, bool valid,
                                             bool keep = true)
{
    const auto at = [&](int i) { return keep ? c[i] * f : 0.0f; };
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t a = pack2<F16>(at(4 * i + 2 * j), at(4 * i + 2 * j + 1));
            const uint32_t b = pack2<F16>(at(4 * i + 4 + 2 * j), at(4 * i + 4 + 2 * j + 1));
            const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
            w[j] = r[0];
            w[2 + j] = r[1];
        }
        if (valid)
            store16<false>(row + 8 * (i + g), w);
    }
}

// The same in fp32.
__device__ __forceinline__ void store_column_f32(float* row, const f32x16& c, float f, int g, bool valid,
                                                 bool keep = true)
{
    const auto at = [&](int i) { return keep ? c[i] * f : 0.0f; };
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (valid)
            *reinterpret_cast<f32x4*>(row + 8 * i + 4 * g) =
                f32x4{at(4 * i), at(4 * i + 1), at(4 * i + 2), at(4 * i + 3)};
}

}  // namespace qkr_attn
