// feed_forward_common.h -- the matrix product that the gated feed-forward
// kernels share: tiles of two operands through a ring of LDS stages, products
// on the matrix cores.  Internal header.
//
// A workgroup computes C[a, b] = sum_k A[a, k] B[b, k] for a tile of A rows and
// a tile of B rows, with a down the registers and b across the lanes of
// v_mfma_f32_32x32x16 (32x32x64 for 8 bits), so that a, the operand of the
// contiguous dimension of the output, leaves 16 bytes of a row in a lane.
//
// An operand's matrix holds k along its rows (kRows: row a of the matrix is row
// a of the operand) or down its rows (kColumns: column a of the matrix is row a
// of the operand).  A stage is 64 bytes of k of kRows (32 numbers of 16 bits, 64
// of 8), or 32 rows of kColumns, laid out in slabs of 32 rows of 64 bytes whose
// 16-byte chunks are permuted as attention_common.h describes: row fragments of
// kRows and transposed reads of kColumns both touch every bank evenly, and 16
// rows of 64 bytes are one load of a wave straight into LDS.  The k of lane 32 g
// + n in a fragment is 8 g .. 8 g + 7 of 16 for both, so that they may be mixed.
//
// The next loads are issued into the slot of a stage when all its fragments have
// been read (of stage s + 4, in a ring of four), and one barrier a stage says both that a slot is free
// and that the next stage is there.  Loads past the last stage read nothing (their
// range is empty) and keep the count of loads in flight the same for every stage.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "attention_common.h"

namespace qkr_ff {

using namespace qkr_attn;

typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

enum Type { kBf16, kFp16, kFp8 };
enum Form { kRows, kColumns };

constexpr int kStageBytes = 64;     // of k, of a row of kRows
constexpr int kStageRows = 32;      // of k, of kColumns
constexpr uint32_t kOutside = 0x80000000u;   // a buffer offset that is out of every range

// One operand's matrix as a workgroup reads it.
struct Matrix {
    const char* at;       // its first row of the tile (kRows), or first column (kColumns)
    int64_t pitch;        // bytes from row to row
    int rows;             // operand rows left from the tile's first one (may be above the tile's)
};

// This lane's and wave's part of loading a tile of one operand: COUNT groups of
// 16 rows by 64 bytes, groups first .. first + COUNT - 1 of the tile.
template <int FORM, int COUNT>
struct Loader {
    uint32_t off[COUNT];
    uint32_t chunk;       // this lane's byte in a row's 64 (kRows)
    uint64_t at;
    uint32_t pitch, last; // last: bytes of the range up to the start of the last row (kRows), or of its columns
    int32_t k;            // bytes (kRows) or rows (kColumns) of k left

    // group_rows: operand rows that the matrix's tile begins before group `first`
    __device__ __forceinline__ Loader(const Matrix& m, int first, int64_t k_size, int lane)
    {
        chunk = ((lane & 3) ^ ((lane >> 4) & 3)) << 4;
        at = reinterpret_cast<uint64_t>(m.at);
        pitch = (uint32_t)m.pitch;
        k = (int32_t)k_size;
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int g = first + i;
            off[i] = chunk + (FORM == kRows ? (uint32_t)((lane >> 2) + 16 * g) * pitch
                                            : (uint32_t)((lane >> 2) + 16 * (g & 1)) * pitch + (g >> 1) * 64);
        }
        last = FORM == kRows ? (uint32_t)(m.rows - 1) * pitch : 2u * (uint32_t)m.rows;
        if (m.rows <= 0)
            k = 0;
    }

    // The next stage's range, for its COUNT calls of load().
    struct Stage {
        u32x4 rsrc;
        uint32_t mask;
    };

    __device__ __forceinline__ Stage next()
    {
        Stage s;
        uint32_t bytes;
        if constexpr (FORM == kRows) {
            const int left = k < kStageBytes ? k : kStageBytes;
            bytes = left > 0 ? last + left : 0;
            s.mask = (int)chunk < left ? 0 : kOutside;
        } else {
            const int left = k < kStageRows ? k : kStageRows;
            bytes = left > 0 ? (uint32_t)(left - 1) * pitch + last : 0;
            s.mask = 0;
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
        __asm__ volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                         : : "v"(FORM == kRows ? off[i] | s.mask : off[i]), "s"(s.rsrc), "s"(scalar(to)) : "memory");
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

// Byte addresses of this lane's part of a tile, slot by slot of the ring.
template <int FORM>
struct FragmentAt {
    uint32_t lane[2];

    __device__ __forceinline__ FragmentAt(uint32_t lds, int ln)
    {
        const int n = ln & 31, g = ln >> 5, l = ln & 15;
        if constexpr (FORM == kRows) {
            lane[0] = lds + n * 64 + ((g ^ ((n >> 2) & 3)) << 4);
            lane[1] = lds + n * 64 + (((2 + g) ^ ((n >> 2) & 3)) << 4);
        } else {
            const int r = 8 * g + (l >> 2), chunk = ((ln >> 4) & 1) * 2 + ((l & 3) >> 1);
            lane[0] = lds + r * 64 + ((chunk ^ (2 * g)) << 4) + (l & 1) * 8;
            lane[1] = lds + (r + 4) * 64 + ((chunk ^ (2 * g + 1)) << 4) + (l & 1) * 8;
        }
    }

    // Operand rows 32 i .. 32 i + 31 of the tile, k step kk of the stage; `off`: the
    // slot's and the tile's offset.
    __device__ __forceinline__ u32x4 read(uint32_t off, int i, int kk) const
    {
        if constexpr (FORM == kRows) {
            return *reinterpret_cast<LdsVec>(lane[kk] + off + i * kSlab);
        } else {
            const uint32_t o = off + i * kSlab + kk * 1024;
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                reinterpret_cast<LdsQuad>(lane[0] + o)));
            const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                reinterpret_cast<LdsQuad>(lane[1] + o)));
            return u32x4{a[0], a[1], b[0], b[1]};
        }
    }
};

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

template <int T>
struct Fragment {                   // 16 numbers of 16 bits, or 64 of 8, of a row's k
    u32x4 v[T == kFp8 ? 2 : 1];
};

template <int T>
__device__ __forceinline__ f32x16 product(const Fragment<T>& a, const Fragment<T>& b, f32x16 c)
{
    if constexpr (T == kFp8) {
        const i32x8 x = __builtin_bit_cast(i32x8, a), y = __builtin_bit_cast(i32x8, b);
        // both operands e4m3 (0), no block scales (all 1: 2^(127 - 127)); it aligns runs
        // of eight products to their largest (feed_forward.h), at twice the rate of 16 bits
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
    } else {
        return mfma<T == kFp16>(a.v[0], b.v[0], c);
    }
}

// What a group of WA x WB waves computes: NA x NB blocks of 32 x 32 a wave.  With
// PAIRED the A tile is two halves, of two matrices, and so is a wave's part of it:
// its first NA / 2 blocks are of the one, the others the same rows of the other.
// A group is a workgroup, or one wave, which waits for no other.
// STAGES: slots of the ring.
template <int T, int FORM_A, int FORM_B, bool PAIRED, int NA, int NB, int WA, int WB, int STAGES = 4>
struct Product {
    static constexpr int kStages = STAGES;
    static constexpr int kWaves = WA * WB;
    static constexpr int kRowsA = 32 * NA * WA, kRowsB = 32 * NB * WB;
    static constexpr int kLoadsA = kRowsA / 16 / kWaves, kLoadsB = kRowsB / 16 / kWaves;
    static constexpr int kTileA = kRowsA * 64, kSlot = (kRowsA + kRowsB) * 64;
    static constexpr int kLds = kStages * kSlot;
    static_assert(kLoadsA * kWaves * 16 == kRowsA && kLoadsB * kWaves * 16 == kRowsB, "whole groups a wave");
    static_assert(!PAIRED || NA % 2 == 0, "a pair of blocks");
    // one wave loads both halves of a pair
    using LoadA = std::conditional_t<PAIRED && kWaves == 1, PairLoader<FORM_A, kLoadsA>, Loader<FORM_A, kLoadsA>>;
    using LoadB = Loader<FORM_B, kLoadsB>;

    f32x16 c[NA][NB];

    struct Fragments {
        Fragment<T> a[NA], b[NB];
    };

    // The block of a wave's ith, from the wave's first one.
    static constexpr int block_a(int i) { return PAIRED && i >= NA / 2 ? i - NA / 2 + NA * WA / 2 : i; }
    static constexpr int first_a(int wave) { return wave % WA * (PAIRED ? NA / 2 : NA); }
    static constexpr int first_b(int wave) { return wave / WA * NB; }

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                c[i][j] = f32x16{};
    }

    // Block (i, j), fetched from where the sums are kept when it is asked for.
    __device__ __forceinline__ f32x16 block(int i, int j)
    {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (NA * NB >= 16)
            __asm__ volatile("" : "+a"(c[i][j]));
        return c[i][j];
    }

    // N of this wave's loads may be in flight, its LDS reads are done, and all waves are here.
    template <int N>
    static __device__ __forceinline__ void wait()
    {
        if constexpr (kWaves > 1)
            __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
        else
            __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
    }

    // Adds `stages` (1 or more) stages of the two loaders' matrices.  The kLds bytes at `lds` are
    // free at the start and at the end.
    __device__ __forceinline__ void add(LoadA& la, LoadB& lb, int stages, uint32_t lds, int wave, int lane)
    {
        const FragmentAt<FORM_A> fa(lds + first_a(wave) * kSlab, lane);
        const FragmentAt<FORM_B> fb(lds + kTileA + first_b(wave) * kSlab, lane);
        const uint32_t to_a = lds + wave * kLoadsA * 1024, to_b = lds + kTileA + wave * kLoadsB * 1024;
        uint32_t fill = 0, slot = 0;
        constexpr int kLoads = kLoadsA + kLoadsB, kReads = NA + NB, kProducts = NA * NB;
        const auto after = [](uint32_t at) { return at == kLds - kSlot ? 0 : at + kSlot; };
        const auto read = [&](Fragments& f, int r, int kk) {       // b's after a's first: the order of use
            Fragment<T>& to = r == 0 ? f.a[0] : r <= NB ? f.b[r - 1] : f.a[r - NB];
#pragma unroll
            for (int h = 0; h < (T == kFp8 ? 2 : 1); ++h) {
                const int step = T == kFp8 ? h : kk;
                to.v[h] = r == 0 ? fa.read(slot, block_a(0), step)
                          : r <= NB ? fb.read(slot, r - 1, step)
                                    : fa.read(slot, block_a(r - NB), step);
            }
        };
        // The products of f, under which the fragments of the next step are read and,
        // with LOADS, the next stage's loads issued; in this order, a few between two
        // products, which take 32 cycles each (64 in 8 bits) and run on by themselves.
        const auto multiply = [&](const Fragments& f, Fragments& next, int kk, auto loads) {
            constexpr bool LOADS = decltype(loads)::value;
            typename LoadA::Stage sa;
            typename LoadB::Stage sb;
            if constexpr (LOADS) {
                sa = la.next();
                sb = lb.next();
            }
#pragma unroll
            for (int t = 0; t < kProducts; ++t) {
#pragma unroll
                for (int r = t * kReads / kProducts; r < (t + 1) * kReads / kProducts; ++r)
                    read(next, r, kk);
                if constexpr (LOADS) {
#pragma unroll
                    for (int q = t * kLoads / kProducts; q < (t + 1) * kLoads / kProducts; ++q) {
                        if (q < kLoadsA)
                            la.load(sa, q, to_a + fill + q * 1024);
                        else
                            lb.load(sb, q - kLoadsA, to_b + fill + (q - kLoadsA) * 1024);
                    }
                }
                c[t / NB][t % NB] = product<T>(f.a[t / NB], f.b[t % NB], c[t / NB][t % NB]);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (LOADS)
                fill = after(fill);
        };
        // The sums of the large tiles take half of a lane's registers, the half that
        // only the matrix cores reach: said here, or some are spilled.
        const auto keep = [&] {
            if constexpr (kProducts >= 16) {
#pragma unroll
                for (int t = 0; t < kProducts; ++t)
                    __asm__ volatile("" : "+a"(c[t / NB][t % NB]));
            }
        };
        const auto turn = [&] {          // the next stage is there, and the present slot free
            wait<(kStages - 2) * kLoads>();
            slot = after(slot);
        };
        Fragments f0, f1;
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
            const auto sa = la.next();
            const auto sb = lb.next();
#pragma unroll
            for (int q = 0; q < kLoadsA; ++q)
                la.load(sa, q, to_a + fill + q * 1024);
#pragma unroll
            for (int q = 0; q < kLoadsB; ++q)
                lb.load(sb, q, to_b + fill + q * 1024);
            fill = after(fill);
        }
        wait<(kStages - 1) * kLoads>();
#pragma unroll
        for (int r = 0; r < kReads; ++r)
            read(f0, r, 0);
        int s = 0;
        if constexpr (T == kFp8) {
            do {                                         // a stage of zeros at the end of an odd number
                turn();
                multiply(f0, f1, 0, Flag<true>{});
                turn();
                multiply(f1, f0, 0, Flag<true>{});
                keep();
                s += 2;
            } while (s < stages);
        } else {
            do {
                multiply(f0, f1, 1, Flag<false>{});
                turn();
                multiply(f1, f0, 0, Flag<true>{});
                keep();
            } while (++s < stages);
        }
        wait<0>();
    }
};

// Stores a C block's lane (row b, columns a0 .. a0 + 31 of the output at `row`),
// of which `left` columns are there.
template <bool F16>
__device__ __forceinline__ void store_block(uint16_t* row, const f32x16& c, int g, bool valid, int left)
{
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t a = pack2<F16>(c[4 * i + 2 * j], c[4 * i + 2 * j + 1]);
            const uint32_t b = pack2<F16>(c[4 * i + 4 + 2 * j], c[4 * i + 4 + 2 * j + 1]);
            const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
            w[j] = r[0];
            w[2 + j] = r[1];
        }
        if (valid && 8 * (i + g) < left)
            store16<false>(row + 8 * (i + g), w);
    }
}

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
