// gated_feed_forward.hip -- h = act(x W_gate^T) * (x W_up^T) for gfx950 (see
// feed_forward.h).
//
// One product with the rows of both weights as one operand: a wave holds the same
// rows of W_gate and of W_up (feed_forward_common.h), so that gate and up of an
// element end in the same place of two accumulators, and the activation and the
// product are its epilogue.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "feed_forward.h"
#include "feed_forward_common.h"
#include "feed_forward_host.h"

namespace {

using namespace qkr_ff;

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

struct FwdParams {
    const char *x, *w_gate, *w_up;
    const float *x_scale, *gate_scale, *up_scale;
    uint16_t *h, *gate, *up;
    int64_t rows;
    int32_t inner;
    int32_t k_bytes;                  // of a row of x and of the weights
    uint32_t row_tiles, inner_tiles;  // of the grid
};

// The epilogue of a wave's sums: rows from r0 on, columns from i0 on.  Two blocks of
// columns leave as rows of 128 bytes, whole lines, through the wave's `own` 12 KB of
// LDS, 32 rows of each matrix at a time; one block, whose rows are half a line, leaves
// from the registers.  (4608 rows of 6144, 16384 columns, gate and up kept: 1455 us
// from the registers, 1412 so; of 8 bits, whose lanes hold quarters of a line, 902 and
// 747; without gate and up within 1%.)
template <int T, bool F16, int ACT, int BLOCKS, typename P>
__device__ __forceinline__ void finish(const FwdParams& p, P& c, int64_t r0, int i0, int lane, char* own)
{
    constexpr int kRowRuns = T == kFp8 ? P::kPieces / 2 : 1;         // rows of a lane that have a scale
    // all scales at once: one wait for memory
    float s[kRowRuns];
    f32x4 gs[BLOCKS][2][2], us[BLOCKS][2][2];
    if constexpr (T == kFp8) {
#pragma unroll
        for (int q = 0; q < kRowRuns; ++q) {
            const int64_t r = r0 + P::piece_row(2 * q, lane);
            s[q] = r < p.rows ? p.x_scale[r] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int a = i0 + 32 * i + P::piece_column(k / 2, lane, k % 2);
                gs[i][k / 2][k % 2] = us[i][k / 2][k % 2] = f32x4{};
                if (a < p.inner) {
                    gs[i][k / 2][k % 2] = *reinterpret_cast<const f32x4u*>(p.gate_scale + a);
                    us[i][k / 2][k % 2] = *reinterpret_cast<const f32x4u*>(p.up_scale + a);
                }
            }
    }
    const auto projections = [&](auto block, auto piece, float (&gate)[8], float (&up)[8])
                                 __attribute__((always_inline)) {
        constexpr int i = decltype(block)::value, q = decltype(piece)::value;
        c.template piece<i, q>(gate);
        c.template piece<i + BLOCKS, q>(up);
        if constexpr (T == kFp8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                gate[k] *= s[q / 2] * gs[i][q % 2][k / 4][k % 4];
                up[k] *= s[q / 2] * us[i][q % 2][k / 4][k % 4];
            }
        }
    };
    if constexpr (BLOCKS == 1) {
        unrolled<P::kPieces>([&](auto number) __attribute__((always_inline)) {
            constexpr int q = decltype(number)::value;
            const int64_t r = r0 + P::piece_row(q, lane);
            const bool valid = r < p.rows;
            const int left = p.inner - i0;
            const int64_t at = r * p.inner + i0;
            float gate[8], up[8];
            projections(Flag<0>{}, number, gate, up);
            if (p.gate) {
                P::template store_piece<F16>(p.gate + at, gate, q, lane, valid, left);
                P::template store_piece<F16>(p.up + at, up, q, lane, valid, left);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                gate[k] = activated<ACT>(gate[k]) * up[k];
            P::template store_piece<F16>(p.h + at, gate, q, lane, valid, left);
        });
    } else {
        static_assert(BLOCKS == 2 && P::kPieces == 4, "64 rows of 128 bytes");
        constexpr int kMatrix = 32 * 128;            // 32 rows of h, gate and up
        unrolled<P::kPieces * BLOCKS>([&](auto number) __attribute__((always_inline)) {
            constexpr int q = decltype(number)::value / BLOCKS, i = decltype(number)::value % BLOCKS;
            float gate[8], up[8];
            projections(Flag<i>{}, Flag<q>{}, gate, up);
            const int row = P::piece_row(q, lane) % 32, chunk = (32 * i + P::packed_column(q, lane)) / 8;
            u32x4* at = reinterpret_cast<u32x4*>(own + row * 128 + ((chunk ^ (row & 7)) << 4));
            if (p.gate) {
                at[kMatrix / 16] = P::template packed<F16>(gate);
                at[2 * kMatrix / 16] = P::template packed<F16>(up);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                gate[k] = activated<ACT>(gate[k]) * up[k];
            at[0] = P::template packed<F16>(gate);
            if constexpr (q % 2 == 1 && i == BLOCKS - 1) {
                __asm__ volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // the wave's own rows only
                const auto leave = [&](uint16_t* out, int from) __attribute__((always_inline)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int in = 8 * k + lane / 8, c8 = lane % 8;
                        const int64_t r = r0 + q / 2 * 32 + in;
                        const u32x4 w = *reinterpret_cast<const u32x4*>(own + from + in * 128 + ((c8 ^ (in & 7)) << 4));
                        if (r < p.rows && i0 + 8 * c8 < p.inner)
                            store16<false>(out + r * p.inner + i0 + 8 * c8, w);
                    }
                };
                if (p.gate) {
                    leave(p.gate, kMatrix);
                    leave(p.up, 2 * kMatrix);
                }
                leave(p.h, 0);
                __asm__ volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // read before they are written again
            }
        });
    }
}

// Tiles of kRowsB rows of x and kRowsA / 2 columns of h.  Bound by the matrix cores at
// the clock that the card's power leaves: 32760 rows of 5120, 13824 columns, gate and
// up kept, 6.80 ms (1360 TFLOP/s; the library's product of these sizes alone 6.72), and
// 4608 rows of 6144 and 16384 columns in 8 bits 0.69 (2690; 0.62).
template <int T, bool F16, int ACT, int NA, int NB, int WA, int WB>
__global__ __launch_bounds__(64 * WA * WB, 2)
void gated_feed_forward_kernel(const FwdParams p)
{
    using P = Product<T, kRows, kRows, true, NA, NB, WA, WB>;
    __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const TileOf tile(blockIdx.x, p.row_tiles, p.inner_tiles, 4);
    const int64_t r0 = (int64_t)tile.row * P::kRowsB;
    constexpr int kColumnsOf = P::kRowsA / 2;
    const int i0 = tile.column * kColumnsOf;
    const int64_t rows_left = p.rows - r0;
    constexpr int kHalf = WA * WB / 2;
    const int of_up = wave >= kHalf;             // the first half of the waves load W_gate's rows
    const Matrix w = {(of_up ? p.w_up : p.w_gate) + (int64_t)i0 * p.k_bytes, p.k_bytes,
                      p.inner - i0 < kColumnsOf ? p.inner - i0 : kColumnsOf};
    const Matrix x = {p.x + r0 * p.k_bytes, p.k_bytes, rows_left < P::kRowsB ? (int)rows_left : P::kRowsB};
    typename P::LoadA la(w, (wave - of_up * kHalf) * P::kLoadsA, p.k_bytes, lane);
    typename P::LoadB lb(x, wave * P::kLoadsB, p.k_bytes, lane);
    P c;
    c.clear();
    c.add(la, lb, (p.k_bytes + kStageBytes - 1) / kStageBytes, lds_address(lds), wave, lane);
    finish<T, F16, ACT, NA / 2>(p, c, r0 + 32 * P::first_b(wave), i0 + 32 * P::first_a(wave), lane,
                                lds + wave * 12288);
}

// Up to 32 rows of x: the call waits for the weights.  A workgroup takes 32 columns
// of h, its waves a share of k each, through slots of their own (no barriers), and
// the first wave adds their sums in order.  One row of 5120 and 13824 columns: 44.0 us,
// 283 MB of weights at 6.4 TB/s.  Calls of it and of 128 x 128 tiles: one row 53 and 58
// us, 32 rows 59 and 58; of 1536 and 4096 columns 9.5 and 14.3 us, one row as 32.
constexpr int kFewRows = 32, kFewColumns = 32, kFewWaves = 2;

template <int T, bool F16, int ACT>
__global__ __launch_bounds__(64 * kFewWaves, 1)
void gated_feed_forward_few_kernel(const FwdParams p)
{
    using P = Product<T, kRows, kRows, true, 2, 1, 1, 1>;
    constexpr int kRing = P::kLds;
    __shared__ __attribute__((aligned(1024))) char lds[kFewWaves * kRing];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int i0 = (int)blockIdx.x * kFewColumns;
    const int stages = (p.k_bytes + kStageBytes - 1) / kStageBytes, each = (stages + kFewWaves - 1) / kFewWaves;
    const int k0 = wave * each * kStageBytes;
    const int k_left = p.k_bytes - k0 < each * kStageBytes ? p.k_bytes - k0 : each * kStageBytes;
    const int columns = p.inner - i0 < kFewColumns ? p.inner - i0 : kFewColumns;
    const int64_t w0 = (int64_t)i0 * p.k_bytes + k0;
    const uint32_t ring = lds_address(lds) + wave * kRing;
    P c;
    c.clear();
    if (k_left > 0) {
        // one load of 32 rows of W_gate, one of W_up
        typename P::LoadA la(Matrix{p.w_gate + w0, p.k_bytes, columns}, Matrix{p.w_up + w0, p.k_bytes, columns}, k_left,
                             lane);
        typename P::LoadB lb(Matrix{p.x + k0, p.k_bytes, (int)p.rows}, 0, k_left, lane);
        c.add(la, lb, (k_left + kStageBytes - 1) / kStageBytes, ring, 0, lane);
    }
    // (a wave's slots are free for its sums)
    float* sums = reinterpret_cast<float*>(lds + wave * kRing) + lane;
    constexpr int kEach = P::kSide * P::kSide / 64;
    const auto sum = [&](int n) __attribute__((always_inline)) -> auto& {
        return c.c[n / kEach / P::kTilesB][n / kEach % P::kTilesB];
    };
    if (wave > 0) {
#pragma unroll
        for (int n = 0; n < 32; ++n)
            sums[64 * n] = sum(n)[n % kEach];
    }
    __syncthreads();
    if (wave > 0)
        return;
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w)
#pragma unroll
        for (int n = 0; n < 32; ++n)
            sum(n)[n % kEach] += sums[w * (kRing / 4) + 64 * n];
    finish<T, F16, ACT, 1>(p, c, 0, i0, lane, lds);
}

using Fn = void (*)(FwdParams);

template <int T, bool F16, int NA, int NB>
Fn select(int activation)
{
    if constexpr (NA == 0)
        return activation == DIT_FF_SILU ? gated_feed_forward_few_kernel<T, F16, 0>
                                         : gated_feed_forward_few_kernel<T, F16, 1>;
    else
        return activation == DIT_FF_SILU ? gated_feed_forward_kernel<T, F16, 0, NA, NB, 2, NA>
                                         : gated_feed_forward_kernel<T, F16, 1, NA, NB, 2, NA>;
}

// NA, NB: blocks of a wave's tile, or 0 for few rows.
template <int NA, int NB>
Fn select(int dtype, int out_dtype, int activation)
{
    if (dtype == DIT_FF_E4M3)
        return out_dtype == QKR_FP16 ? select<kFp8, true, NA, NB>(activation) : select<kFp8, false, NA, NB>(activation);
    return dtype == QKR_FP16 ? select<kFp16, true, NA, NB>(activation) : select<kBf16, false, NA, NB>(activation);
}

}  // namespace

extern "C" int dit_gated_feed_forward(const dit_ff_args* args, const void* x, const void* w_gate,
                                      const void* w_up, const float* x_scale, const float* gate_scale,
                                      const float* up_scale, void* h, void* gate, void* up,
                                      void* stream)
{
    using namespace qkr_ff_host;
    const int rc = check_args(args, true);
    if (rc != QKR_OK)
        return rc;
    const dit_ff_args& a = *args;
    const bool fp8 = a.dtype == DIT_FF_E4M3;
    if (a.rows == 0)
        return QKR_OK;
    if (!x || !w_gate || !w_up || !h || !gate != !up || (fp8 && (!x_scale || !gate_scale || !up_scale)))
        return QKR_ERR_NULL;
    if (!fp8 && (x_scale || gate_scale || up_scale))
        return QKR_ERR_ARG;
    const uint64_t size = fp8 ? 1 : 2, hidden = a.hidden, inner = a.inner, rows = a.rows;
    const Buffer in[] = {{x, rows * hidden * size, 16}, {w_gate, inner * hidden * size, 16},
                         {w_up, inner * hidden * size, 16}, {x_scale, x_scale ? rows * 4 : 0, 4},
                         {gate_scale, gate_scale ? inner * 4 : 0, 4}, {up_scale, up_scale ? inner * 4 : 0, 4}};
    const Buffer out[] = {{h, rows * inner * 2, 16}, {gate, gate ? rows * inner * 2 : 0, 16},
                          {up, up ? rows * inner * 2 : 0, 16}};
    const int bad = check_buffers(in, 6, out, 3);
    if (bad != QKR_OK)
        return bad;

    FwdParams p = {};
    p.x = static_cast<const char*>(x);
    p.w_gate = static_cast<const char*>(w_gate);
    p.w_up = static_cast<const char*>(w_up);
    p.x_scale = x_scale;
    p.gate_scale = gate_scale;
    p.up_scale = up_scale;
    p.h = static_cast<uint16_t*>(h);
    p.gate = static_cast<uint16_t*>(gate);
    p.up = static_cast<uint16_t*>(up);
    p.rows = a.rows;
    p.inner = a.inner;
    p.k_bytes = a.hidden * (int32_t)size;
    if (a.rows <= kFewRows)
        return launch(select<0, 0>(a.dtype, a.out_dtype, a.activation), (a.inner + kFewColumns - 1) / kFewColumns, p,
                      stream, 64 * kFewWaves);
    const Cut cut = cut_of(a.rows, 2 * (int64_t)a.inner, (p.k_bytes + 127) / 128, false);
    p.row_tiles = (uint32_t)cut.row_tiles;
    p.inner_tiles = (uint32_t)((a.inner + (cut.large ? 127 : 63)) / (cut.large ? 128 : 64));
    const Fn fn = cut.large ? select<4, 2>(a.dtype, a.out_dtype, a.activation)
                        : select<2, 2>(a.dtype, a.out_dtype, a.activation);
    return launch(fn, (int64_t)p.row_tiles * p.inner_tiles, p, stream, cut.large ? 512 : 256);
}
