// feed_forward_common.h -- the matrix product that the gated feed-forward
// kernels share: tiles of two operands through a ring of LDS stages, products
// on the matrix cores.  Internal header.
//
// A workgroup computes C[a, b] = sum_k A[a, k] B[b, k] for a tile of A rows and
// a tile of B rows, with a down the registers and b across the lanes of
// v_mfma_f32_16x16x32 (32x32x64 for 8 bits), so that a, the operand of the
// contiguous dimension of the output, leaves 8 bytes of a row in a lane.  (What a
// large product may take is bounded by the card's power: on random numbers loops of
// the 16x16x32 instruction alone reach 2040 TFLOP/s, of 32x32x16 1730.)
//
// An operand's matrix holds k along its rows (kRows: row a of the matrix is row a
// of the operand) or down its rows (kColumns: column a of the matrix is row a of
// the operand).  A stage is 128 bytes of k of kRows (64 numbers of 16 bits, 128 of
// 8), or 64 rows of k of kColumns.  In LDS both are rows of 128 bytes: the operand
// rows of kRows, or slabs of 64 columns of the 64 rows of kColumns.  A load of a
// wave, straight into LDS, is 8 such rows: whole lines of the L2, whose requests
// are what bounds a tile's loads (rows of 64 bytes, twice as many requests, ran
// 256 x 256 tiles at 1200 TFLOP/s).
//
// 16-byte chunk c of row r is stored at c ^ f(r), where f has 4 for bit 1 of r, 3 for
// bit 2 and 2 for bit 3, exclusively or.  Of a read of 16 bytes a lane, lanes 0-3,
// 12-15 and 20-27 (and so on) are served together: f(6) = 1 lets rows 0-3 and 12-15
// of one chunk and rows 4-11 of the next touch every bank once.  So do rows r .. r + 3
// and r + 8 .. r + 11 of two chunks, which a transposed read takes.  The k of a
// fragment's lane is a run of 8 for both forms, so that they may be mixed.
//
// A stage is two steps of products; while one runs, the fragments of the next are
// read.  LDS is a ring of five slots of a tile, for A and B of a stage in turn: two
// stages and A of a third.  When the fragments of a stage's last step are read, one
// barrier says that its slots are free and that the next stage is there.  Loads past
// the last stage read nothing: their range is empty.  (Loads that go through registers
// and stores of LDS have longer to arrive, but the stores cost more than that gains.)
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>
#include <utility>

#include "attention_common.h"

namespace qkr_ff {

using namespace qkr_attn;

typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

enum Type { kBf16, kFp16, kFp8 };
enum Form { kRows, kColumns };

constexpr int kStageBytes = 128;    // of k, of a row of kRows
constexpr int kStageRows = 64;      // of k, of kColumns
constexpr int kGroupRows = 8;       // LDS rows that a wave loads at a time
constexpr int kSlabBytes = 64 * 128;
constexpr uint32_t kOutside = 0x80000000u;   // a buffer offset that is out of every range

// One operand's matrix as a workgroup reads it.
struct Matrix {
    const char* at;       // its first row of the tile (kRows), or first column (kColumns)
    int64_t pitch;        // bytes from row to row
    int rows;             // operand rows left from the tile's first one (may be above the tile's)
};

// f(r) above, of r / 2.
__device__ __forceinline__ uint32_t swizzle(uint32_t half_row)
{
    return (half_row & 1 ? 4 : 0) ^ (half_row & 2 ? 3 : 0) ^ (half_row & 4 ? 2 : 0);
}

// This lane's and wave's part of loading a tile of one operand: COUNT groups of 8
// LDS rows, groups first .. first + COUNT - 1 of the tile.
template <int FORM, int COUNT>
struct Loader {
    uint32_t off[2];      // of groups of even and odd number, less what follows from the number
    uint32_t chunk[2];    // this lane's byte in a row's 128 (kRows)
    uint64_t at;
    uint32_t pitch, last; // last: bytes of the range up to the start of the last row (kRows), or of its columns
    int32_t k;            // bytes (kRows) or rows (kColumns) of k left

    __device__ __forceinline__ Loader(const Matrix& m, int first, int64_t k_size, int lane)
    {
        at = reinterpret_cast<uint64_t>(m.at);
        pitch = (uint32_t)m.pitch;
        k = (int32_t)k_size;
        static_assert(COUNT % 2 == 0 && (FORM == kRows || COUNT == 2 || COUNT == 4 || COUNT % 8 == 0), "whole slabs");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            chunk[i] = ((lane & 7) ^ swizzle(4 * i + (lane >> 4))) << 4;
            const uint32_t g = first;          // of 8 groups of a slab, slab first / 8
            off[i] = chunk[i] + (FORM == kRows ? ((lane >> 3) + kGroupRows * g) * pitch
                                               : ((lane >> 3) + kGroupRows * (g & 7)) * pitch + (g >> 3) * 128);
        }
        last = FORM == kRows ? (uint32_t)(m.rows - 1) * pitch : 2u * (uint32_t)m.rows;
        if (m.rows <= 0)
            k = 0;
    }

    // The next stage's range, for its COUNT calls of load().
    struct Stage {
        u32x4 rsrc;
        uint32_t off[2];
    };

    __device__ __forceinline__ Stage next()
    {
        Stage s;
        uint32_t bytes;
        if constexpr (FORM == kRows) {
            const int left = k < kStageBytes ? k : kStageBytes;
            bytes = left > 0 ? last + left : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s.off[i] = (int)chunk[i] < left ? off[i] : kOutside;
        } else {
            const int left = k < kStageRows ? k : kStageRows;
            bytes = left > 0 ? (uint32_t)(left - 1) * pitch + last : 0;
            s.off[0] = off[0];
            s.off[1] = off[1];
        }
        s.rsrc = u32x4{scalar((uint32_t)at), scalar((uint32_t)(at >> 32) & 0xffffu), scalar(bytes), kRawBuffer};
        at += FORM == kRows ? (uint64_t)kStageBytes : (uint64_t)kStageRows * pitch;
        k -= FORM == kRows ? kStageBytes : kStageRows;
        return s;
    }

    // Issues the load of group i to LDS address `to`: assembly, and its no-ops, for
    // the reasons that Stager::dma_row_group of attention_common.h gives.
    __device__ __forceinline__ void load(const Stage& s, int i, uint32_t to) const
    {
        // (an offset outside stays outside: the steps of a tile are below 2^31)
        const uint32_t step = FORM == kRows ? (uint32_t)i * (kGroupRows * pitch)
                                            : (uint32_t)(i & 7) * (kGroupRows * pitch) + (uint32_t)(i >> 3) * 128;
        __asm__ volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                         : : "v"(s.off[i & 1] + step), "s"(s.rsrc), "s"(scalar(to)) : "memory");
    }
};

// The same of a tile of two matrices, half of the groups each.
template <int FORM, int COUNT>
struct PairLoader {
    Loader<FORM, COUNT / 2> one, other;

    struct Stage {
        typename Loader<FORM, COUNT / 2>::Stage one, other;
    };

    __device__ __forceinline__ PairLoader(const Matrix& a, const Matrix& b, int64_t k_size, int lane)
        : one(a, 0, k_size, lane), other(b, 0, k_size, lane)
    {
    }

    __device__ __forceinline__ Stage next() { return Stage{one.next(), other.next()}; }

    __device__ __forceinline__ void load(const Stage& s, int i, uint32_t to) const
    {
        if (i < COUNT / 2)
            one.load(s.one, i, to);
        else
            other.load(s.other, i - COUNT / 2, to);
    }
};

// Byte addresses of this lane's part of a tile.  SIDE: operand rows of a fragment,
// 16 (by 32 numbers of k) or, of kRows, 32 (by 64 numbers of 8 bits, in two reads).
template <int FORM, int SIDE>
struct FragmentAt {
    static_assert(SIDE == 16 || FORM == kRows, "8 bits are kRows");
    static constexpr int kN = SIDE == 16 && FORM == kRows ? 2 : 4;
    uint32_t own[kN], lane[kN];     // in any slot, and in the present one

    __device__ __forceinline__ FragmentAt(uint32_t lds, int ln)
    {
        const int n = ln % SIDE, g = ln / SIDE, l = ln & 15;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            if constexpr (FORM == kRows) {
                // 16: chunks 4 i + g of step i; 32: chunks 2 i + g, two for a step
                own[i] = lds + n * 128 + (((i * (64 / SIDE) + g) ^ swizzle((n >> 1) & 7)) << 4);
            } else {
                // rows 8 g .. 8 g + 3 (+ 4 for odd i) of a step, 16 columns of blocks 2 (i / 2) + 4 m
                const uint32_t r = 8 * g + 4 * (i & 1) + (l >> 2);
                const uint32_t chunk = (i >> 1) * 2 + ((l & 3) >> 1);
                own[i] = lds + r * 128 + ((chunk ^ swizzle((r >> 1) & 7)) << 4) + (l & 1) * 8;
            }
        }
    }

    __device__ __forceinline__ void to(uint32_t slot)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            lane[i] = own[i] + slot;
    }

    // Operand rows SIDE i .. of the tile, chunk set `kk` of the stage.
    __device__ __forceinline__ u32x4 read(int i, int kk) const
    {
        if constexpr (FORM == kRows) {
            return *reinterpret_cast<LdsVec>(lane[kk] + i * (SIDE * 128));
        } else {
            // 4 blocks of 16 columns in a slab: their chunks are 2 (i % 4) and the next
            const uint32_t o = (i >> 2) * kSlabBytes + kk * 4096, flip = (i & 2) ? 64 : 0;
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                reinterpret_cast<LdsQuad>((lane[2 * (i & 1)] ^ flip) + o)));
            const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                reinterpret_cast<LdsQuad>((lane[2 * (i & 1) + 1] ^ flip) + o)));
            return u32x4{a[0], a[1], b[0], b[1]};
        }
    }
};

template <int V>
struct Flag {
    static constexpr int value = V;
};

// f(Flag<0>{}), f(Flag<1>{}) .. N times: a loop of that many products is more than
// the compiler unrolls.
template <int... I, typename F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, I...>, F&& f)
{
    (f(Flag<I>{}), ...);
}

template <int N, typename F>
__device__ __forceinline__ void unrolled(F&& f)
{
    unrolled(std::make_integer_sequence<int, N>{}, f);
}

template <int T>
struct Fragment {                   // 16 rows by 32 numbers of 16 bits, or 32 by 64 of 8
    u32x4 v[T == kFp8 ? 2 : 1];
};

template <int T>
using Sums = std::conditional_t<T == kFp8, f32x16, f32x4>;

// c += a b.  KEPT: c stays where only the matrix cores reach, in assembly, because the
// compiler moves 64 such sums to and fro.  Assembly has to keep the distances itself:
// two wait states after a vector instruction that wrote a or b (a copy, say; reads of
// LDS are waited for), and settle_sums() before the sums are read.
template <int T, bool KEPT>
__device__ __forceinline__ void add_product(const Fragment<T>& a, const Fragment<T>& b, Sums<T>& c)
{
    if constexpr (T == kFp8) {
        const i32x8 x = __builtin_bit_cast(i32x8, a), y = __builtin_bit_cast(i32x8, b);
        // both operands e4m3 (0), no block scales (all 1: 2^(127 - 127)); it aligns runs
        // of eight products to their largest (feed_forward.h), at twice the rate of 16 bits
        c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
    } else if constexpr (KEPT && T == kFp16) {
        __asm__ volatile("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a.v[0]), "v"(b.v[0]));
    } else if constexpr (KEPT) {
        __asm__ volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a.v[0]), "v"(b.v[0]));
    } else if constexpr (T == kFp16) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a.v[0]), __builtin_bit_cast(f16x8, b.v[0]),
                                                   c, 0, 0, 0);
    } else {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v[0]),
                                                    __builtin_bit_cast(bf16x8, b.v[0]), c, 0, 0, 0);
    }
}

// The longest wait of a matrix instruction's result, of which an earlier one has passed.
__device__ __forceinline__ void settle_sums() { __asm__ volatile("s_nop 15\n\ts_nop 7" : : : "memory"); }

// What a group of WA x WB waves computes: NA x NB blocks of 32 x 32 a wave.  With
// PAIRED the A tile is two halves, of two matrices, and so is a wave's part of it:
// its first NA / 2 blocks are of the one, the others the same rows of the other.
// A group is a workgroup, or one wave, which waits for no other.
template <int T, int FORM_A, int FORM_B, bool PAIRED, int NA, int NB, int WA, int WB>
struct Product {
    static constexpr int kWaves = WA * WB;
    static constexpr int kRowsA = 32 * NA * WA, kRowsB = 32 * NB * WB;
    static constexpr int kLoadsA = kRowsA / kGroupRows / kWaves, kLoadsB = kRowsB / kGroupRows / kWaves;
    // LDS: a ring of 5 slots of a tile, for A and B of a stage in turn
    static constexpr int kSlot = 128 * (kRowsA > kRowsB ? kRowsA : kRowsB), kLds = 5 * kSlot;
    static_assert(kLoadsA * kWaves * kGroupRows == kRowsA && kLoadsB * kWaves * kGroupRows == kRowsB,
                  "whole groups a wave");
    static_assert(!PAIRED || NA % 2 == 0, "a pair of blocks");
    // one wave loads both halves of a pair
    using LoadA = std::conditional_t<PAIRED && kWaves == 1, PairLoader<FORM_A, kLoadsA>, Loader<FORM_A, kLoadsA>>;
    using LoadB = Loader<FORM_B, kLoadsB>;

    static constexpr int kSide = T == kFp8 ? 32 : 16;      // of a product's operands
    static constexpr int kTilesA = 32 * NA / kSide, kTilesB = 32 * NB / kSide;

    static constexpr bool kKept = NA * NB >= 8;     // the sums take half of a lane's registers
    Sums<T> c[kTilesA][kTilesB];

    // Fragments of A are read this many rows of products ahead, into a ring.
    static constexpr int kAhead = kTilesA < 4 ? kTilesA - 1 : 3, kRing = kAhead + 1;
    static_assert(kTilesA % kRing == 0, "a fragment's place does not change from step to step");

    // The operand rows (in kSide) of a wave's ith fragment, from the wave's first one.
    static constexpr int tile_a(int i)
    {
        return PAIRED && i >= kTilesA / 2 ? i - kTilesA / 2 + kTilesA * WA / 2 : i;
    }
    // A wave's first blocks of 32.
    static constexpr int first_a(int wave) { return wave % WA * (PAIRED ? NA / 2 : NA); }
    static constexpr int first_b(int wave) { return wave / WA * NB; }
    // ... in bytes of LDS (kColumns: slabs of two blocks, so a wave's first is even)
    static constexpr int bytes_of(int form, int block) { return form == kRows ? block * 4096 : block / 2 * kSlabBytes; }
    static_assert(FORM_A == kRows || (NA % 2 == 0 && !PAIRED), "whole slabs a wave");
    static_assert(FORM_B == kRows || NB % 2 == 0, "whole slabs a wave");

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kTilesA; ++i)
#pragma unroll
            for (int j = 0; j < kTilesB; ++j)
                c[i][j] = Sums<T>{};
    }

    // The sums leave in pieces of 8: piece (i, p), of block i of 32 columns (rows of A)
    // and p of 2 NB, holds for this lane two runs of 4 columns of one row (of B).
    // 16 bits: p is 16 rows; 8 bits: half of the columns of 32 rows.
    static constexpr int kPieces = 2 * NB;
    static __device__ __forceinline__ int piece_row(int p, int lane)
    {
        return T == kFp8 ? p / 2 * 32 + lane % 32 : p * 16 + lane % 16;
    }
    static __device__ __forceinline__ int piece_column(int p, int lane, int run)
    {
        return T == kFp8 ? p % 2 * 16 + run * 8 + lane / 32 * 4 : run * 16 + lane / 16 * 4;
    }

    // Fetched from where the sums are kept when it is asked for, and not before.
    template <int i, int p>
    __device__ __forceinline__ void piece(float (&v)[8])
    {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (T == kFp8) {
            if constexpr (kKept)
                __asm__ volatile("" : "+a"(c[i][p / 2]));
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = c[i][p / 2][8 * (p % 2) + k];
        } else {
            if constexpr (kKept)
                __asm__ volatile("" : "+a"(c[2 * i][p]), "+a"(c[2 * i + 1][p]));
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = c[2 * i + k / 4][p][k % 4];
        }
    }

    // A piece in 16 bits: the lanes that hold neighbouring runs trade them, so that each
    // has 16 bytes of a row, from column packed_column() of the block on.
    template <bool F16>
    static __device__ __forceinline__ u32x4 packed(const float (&v)[8])
    {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t x = pack2<F16>(v[2 * j], v[2 * j + 1]), y = pack2<F16>(v[4 + 2 * j], v[5 + 2 * j]);
            if constexpr (T == kFp8) {
                const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
                w[j] = r[0];
                w[2 + j] = r[1];
            } else {
                const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
                w[j] = r[0];
                w[2 + j] = r[1];
            }
        }
        return w;
    }

    static __device__ __forceinline__ int packed_column(int p, int lane)
    {
        return T == kFp8 ? p % 2 * 16 + lane / 32 * 8 : (lane >> 4 & 1) * 16 + (lane >> 5) * 8;
    }

    // Stores a piece: `row` is block i's first column in the lane's output row, of which
    // `left` columns are there.
    template <bool F16>
    static __device__ __forceinline__ void store_piece(uint16_t* row, const float (&v)[8], int p, int lane, bool valid,
                                                       int left)
    {
        const u32x4 w = packed<F16>(v);
        const int at = packed_column(p, lane);
        if (valid && at < left)
            store16<false>(row + at, w);
    }

    // All but N of this wave's loads and all of its LDS reads are done, and all waves are here.
    template <int N>
    static __device__ __forceinline__ void meet()
    {
        if constexpr (kWaves > 1)
            __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
        else
            __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
    }

    // Adds `stages` (1 or more) stages of the two loaders' matrices.  The kLds bytes at
    // `lds` are free at the start and at the end.
    __device__ __forceinline__ void add(LoadA& la, LoadB& lb, int stages, uint32_t lds, int wave, int lane)
    {
        FragmentAt<FORM_A, kSide> fa(lds + bytes_of(FORM_A, first_a(wave)), lane);
        FragmentAt<FORM_B, kSide> fb(lds + bytes_of(FORM_B, first_b(wave)), lane);
        uint32_t slot_a = 0, slot_b = kSlot;                  // of the present stage
        uint32_t fill_b = 3 * kSlot, fill_a = 4 * kSlot;      // of the loads that are issued now
        const auto advance = [](uint32_t slot) { return slot >= 3 * kSlot ? slot - 3 * kSlot : slot + 2 * kSlot; };
        constexpr int kLoads = kLoadsA + kLoadsB, kProducts = kTilesA * kTilesB;
        constexpr int kSteps = 2;             // of a stage: 32 numbers of k, or 64 of 8 bits
        Fragment<T> a[kRing], b[kSteps][kTilesB];
        const auto read_a = [&](int i, int step) {
#pragma unroll
            for (int h = 0; h < (T == kFp8 ? 2 : 1); ++h)
                a[i % kRing].v[h] = fa.read(tile_a(i), T == kFp8 ? 2 * step + h : step);
        };
        const auto read_b = [&](int j, int step) {
#pragma unroll
            for (int h = 0; h < (T == kFp8 ? 2 : 1); ++h)
                b[step][j].v[h] = fb.read(j, T == kFp8 ? 2 * step + h : step);
        };
        typename LoadA::Stage sa;
        typename LoadB::Stage sb;
        const uint32_t to_a = lds + wave * kLoadsA * 1024, to_b = lds + wave * kLoadsB * 1024;
        // loads 0 .. kLoadsB - 1 of a stage's turn are B's, the others A's of the stage after
        const auto load = [&](int q) __attribute__((always_inline)) {
            if (q == 0)
                sb = lb.next();
            if (q == kLoadsB)
                sa = la.next();
            if (q < kLoadsB)
                lb.load(sb, q, fill_b + to_b + q * 1024);
            else
                la.load(sa, q - kLoadsB, fill_a + to_a + (q - kLoadsB) * 1024);
        };
        // A step's products, row by row of A's fragments, and between them, a few
        // instructions under each (16 cycles, 64 in 8 bits), in this order:
        //   A    the fragment of the row kAhead further (in the last rows, of the next step);
        //   B    the next step's, early;
        //   in a stage's last step, before the first read of the next stage, and once this
        //        wave's reads are done and the next stage is there, the barrier that says so of
        //        all waves;
        //   from there to the next one, at even distances, the loads into the two slots that
        //        this freed: B of the stage after the next, then A of the one after that.  (A
        //        wave waits while its load is taken, so loads in a row hold up its products: all
        //        at once measured 1170 TFLOP/s, over half of a stage 1310.)
        constexpr int kTurn = (kTilesA - kAhead) * kTilesB;
        const auto turn = [&]() __attribute__((always_inline)) {
            meet<kLoadsA>();
            fill_b = slot_a;
            fill_a = slot_b;
            slot_a = advance(slot_a);
            slot_b = advance(slot_b);
            fa.to(slot_a);
            fb.to(slot_b);
        };
        // loads of products 0 .. t - 1 after a turn
        const auto loads_by = [](int t) { return (t * kLoads + 2 * kProducts - 1) / (2 * kProducts); };
        const auto step = [&](auto which) {
            constexpr int kStep = decltype(which)::value;
            constexpr bool LAST = kStep == kSteps - 1;
            constexpr int kFrom = LAST ? kTurn : 0, kSpan = (kProducts - kFrom) / 2 > 0 ? (kProducts - kFrom) / 2 : 1;
            unrolled<kProducts>([&](auto number) __attribute__((always_inline)) {
                constexpr int t = decltype(number)::value, i = t / kTilesB, j = t % kTilesB;
                if constexpr (LAST && t == kTurn)
                    turn();
                if constexpr (j == 0)
                    read_a((i + kAhead) % kTilesA, i + kAhead < kTilesA ? kStep : (kStep + 1) % kSteps);
                if constexpr (t >= kFrom && t < kFrom + kSpan) {
#pragma unroll
                    for (int r = (t - kFrom) * kTilesB / kSpan; r < (t - kFrom + 1) * kTilesB / kSpan; ++r)
                        read_b(r, (kStep + 1) % kSteps);
                }
                constexpr int kSince = LAST ? (t >= kTurn ? t - kTurn : t + 2 * kProducts - kTurn)
                                            : t + kProducts - kTurn;
#pragma unroll
                for (int q = loads_by(kSince); q < loads_by(kSince + 1); ++q)
                    load(q);
                add_product<T, kKept>(a[i % kRing], b[kStep][j], c[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        // A and B of the first stage, A of the second, and what would follow a turn before it
        const auto load_a = [&](uint32_t slot) __attribute__((always_inline)) {
            sa = la.next();
#pragma unroll
            for (int q = 0; q < kLoadsA; ++q)
                la.load(sa, q, slot + to_a + q * 1024);
        };
        constexpr int kBefore = loads_by(kProducts - kTurn);
        load_a(0);
        sb = lb.next();
#pragma unroll
        for (int q = 0; q < kLoadsB; ++q)
            lb.load(sb, q, kSlot + to_b + q * 1024);
        load_a(2 * kSlot);
#pragma unroll
        for (int q = 0; q < kBefore; ++q)
            load(q);
        meet<kLoadsA + kBefore>();
        fa.to(slot_a);
        fb.to(slot_b);
#pragma unroll
        for (int j = 0; j < kTilesB; ++j)
            read_b(j, 0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            read_a(i, 0);
        int s = 0;
        do {
            step(Flag<0>{});
            step(Flag<1>{});
            if constexpr (kKept && T == kFp8) {
#pragma unroll
                for (int i = 0; i < kTilesA; ++i)
#pragma unroll
                    for (int j = 0; j < kTilesB; ++j)
                        __asm__ volatile("" : "+a"(c[i][j]));     // or some are spilled
            }
        } while (++s < stages);
        meet<0>();
        if constexpr (kKept && T != kFp8)
            settle_sums();
    }
};

// The (row of tiles, column of tiles) of hardware block `bid` of rows x columns
// tiles: each die walks one run of them, in bands of `band` rows of tiles, column
// by column, so that the tiles that run on it at a time share both operands in
// its L2.
struct TileOf {
    int row, column;

    __device__ __forceinline__ TileOf(uint32_t bid, uint32_t rows, uint32_t columns, uint32_t band)
    {
        const uint32_t at = (uint32_t)logical_block<-1>(bid, rows * columns);
        const uint32_t whole = at / (band * columns), first = whole * band;
        const uint32_t height = rows - first < band ? rows - first : band;
        const uint32_t in = at - first * columns;
        row = first + in % height;
        column = in / height;
    }
};

// z and dz/dx of the activations y = x / (1 + exp(-z)): SiLU (z = x), and GELU by
// its tanh, 0.5 x (1 + tanh(w)) with w = sqrt(2 / pi) (x + 0.044715 x^3), which
// is the same with z = 2 w.
template <int ACT>
__device__ __forceinline__ float activation_z(float x)
{
    return ACT == 0 ? x : 1.5957691216057308f * x * __builtin_fmaf(0.044715f * x, x, 1.0f);
}

__device__ __forceinline__ float logistic(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

template <int ACT>
__device__ __forceinline__ float activated(float x) { return x * logistic(activation_z<ACT>(x)); }

// The activation and its derivative s + x s (1 - s) dz/dx.
template <int ACT>
__device__ __forceinline__ void activated(float x, float& y, float& slope)
{
    const float s = logistic(activation_z<ACT>(x));
    y = x * s;
    if constexpr (ACT == 0) {
        slope = __builtin_fmaf(y, 1.0f - s, s);
    } else {
        // beyond 64 either s or 1 - s is 0, and the square must not become infinite
        const float b = __builtin_amdgcn_fmed3f(x, -64.0f, 64.0f);
        slope = __builtin_fmaf(y * (1.0f - s), 1.5957691216057308f * __builtin_fmaf(3 * 0.044715f * b, b, 1.0f), s);
    }
}

}  // namespace qkr_ff
