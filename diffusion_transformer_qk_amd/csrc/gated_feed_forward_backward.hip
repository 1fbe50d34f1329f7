// gated_feed_forward_backward.hip -- dx, dw_gate and dw_up for gfx950 (see
// feed_forward.h).
//
// First dgate and dup, element by element from dh, gate and up, into the
// workspace; then two products (feed_forward_common.h), each of both halves at
// once:
//   dx = dgate W_gate + dup W_up: one sum over 2 * inner, the weights read down
//        their rows by transposed reads of LDS;
//   dw = dgate^T x and dup^T x: sums over the rows, both operands read down.
// Kept gate and up cost 4 bytes an element and a pass; computing them again would
// cost half as many products as the two above.
//
// fp16: dgate and dup are stored times a power of two that brings the largest of
// them just below 2^15; a pass before finds it (the tensors are read once more,
// a few hundredths of the products' time).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "feed_forward.h"
#include "feed_forward_common.h"
#include "feed_forward_host.h"

namespace {

using namespace qkr_ff;

struct BwdParams {
    const uint16_t *dh, *x, *w_gate, *w_up, *gate, *up;
    uint16_t *dx, *dw_gate, *dw_up;
    uint16_t* d;              // [2][rows][inner]: dgate and dup
    float* largest;           // fp16: [largest_blocks] largest finite |dgate|, |dup|
    uint32_t largest_blocks;
    int64_t rows;
    int32_t hidden, inner;
    uint32_t row_tiles, column_tiles;   // of the grid
};

constexpr int kThreads = 256;

// The power of two that dgate and dup are divided by: the largest becomes 2^14 .. 2^15.
__device__ __forceinline__ int stored_exponent(const BwdParams& p, float* slot)
{
    float top = 0.0f;
    for (uint32_t i = threadIdx.x; i < p.largest_blocks; i += kThreads)
        top = fmaxf(top, p.largest[i]);
    top = block_max<4>(top, slot);
    return top > 0.0f ? __builtin_amdgcn_frexp_expf(top) - 15 : 0;
}

// dgate and dup of 8 elements.
template <bool F16, int ACT>
__device__ __forceinline__ void gradients(const BwdParams& p, int64_t i, float (&dgate)[8], float (&dup)[8])
{
    float dh[8], gate[8], up[8];
    unpack8<F16>(load16<true>(p.dh + i), dh);
    unpack8<F16>(load16<true>(p.gate + i), gate);
    unpack8<F16>(load16<true>(p.up + i), up);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float y, slope;
        activated<ACT>(gate[k], y, slope);
        dgate[k] = dh[k] * up[k] * slope;
        dup[k] = dh[k] * y;
    }
}

// An infinity or NaN is lost whatever scales it, and must not unscale the others.
__device__ __forceinline__ float finite(float v) { return fabsf(v) <= 0x1.fffffep127f ? fabsf(v) : 0.0f; }

template <int ACT>
__global__ __launch_bounds__(kThreads)
void feed_forward_largest_kernel(const BwdParams p)
{
    __shared__ float slot[4];
    const int64_t n = p.rows * p.inner;
    float top = 0.0f;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kVec; i < n;
         i += (int64_t)gridDim.x * kThreads * kVec) {
        float a[8], b[8];
        gradients<true, ACT>(p, i, a, b);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            top = fmaxf(top, fmaxf(finite(a[k]), finite(b[k])));
    }
    top = block_max<4>(top, slot);
    if (threadIdx.x == 0)
        p.largest[blockIdx.x] = top;
}

template <bool F16, int ACT>
__global__ __launch_bounds__(kThreads)
void feed_forward_gradients_kernel(const BwdParams p)
{
    __shared__ float slot[4];
    const int64_t n = p.rows * p.inner;
    int e = 0;
    if constexpr (F16)
        e = stored_exponent(p, slot);
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kVec; i < n;
         i += (int64_t)gridDim.x * kThreads * kVec) {
        float a[8], b[8];
        gradients<F16, ACT>(p, i, a, b);
        if constexpr (F16) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                a[k] = __builtin_amdgcn_ldexpf(a[k], -e);
                b[k] = __builtin_amdgcn_ldexpf(b[k], -e);
            }
        }
        store16<false>(p.d + i, pack8<F16>(a));
        store16<false>(p.d + n + i, pack8<F16>(b));
    }
}

// A wave's sums times 2^e, to rows from r0 on (of `rows`) and columns from a0 on of
// [rows, columns] at `out`.
template <bool F16, typename P>
__device__ __forceinline__ void store(P& c, uint16_t* out, int64_t r0, int64_t rows, int a0, int columns, int e,
                                      int lane)
{
    constexpr int kBlocks = P::kTilesA * P::kSide / 32;
    unrolled<P::kPieces * kBlocks>([&](auto number) __attribute__((always_inline)) {
        constexpr int q = decltype(number)::value / kBlocks, i = decltype(number)::value % kBlocks;
        const int64_t r = r0 + P::piece_row(q, lane);
        float v[8];
        c.template piece<i, q>(v);
        if constexpr (F16) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = __builtin_amdgcn_ldexpf(v[k], e);
        }
        const int a = a0 + 32 * i;
        P::template store_piece<F16>(out + r * columns + a, v, q, lane, r < rows, columns - a);
    });
}

// Tiles of kRowsB rows and kRowsA columns of dx.
template <bool F16, int N>
__global__ __launch_bounds__(256, N == 4 ? 1 : 2)
void feed_forward_dx_kernel(const BwdParams p)
{
    using P = Product<F16 ? kFp16 : kBf16, kColumns, kRows, false, N, N, 2, 2>;
    __shared__ __attribute__((aligned(2 * P::kSlot))) char lds[P::kLds];
    __shared__ float slot[4];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const TileOf tile(blockIdx.x, p.row_tiles, p.column_tiles, 8);
    const int64_t r0 = (int64_t)tile.row * P::kRowsB, rows_left = p.rows - r0;
    const int h0 = tile.column * P::kRowsA;
    const int rows = rows_left < P::kRowsB ? (int)rows_left : P::kRowsB;
    const int columns = p.hidden - h0 < P::kRowsA ? p.hidden - h0 : P::kRowsA;
    P c;
    c.clear();
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const Matrix w = {reinterpret_cast<const char*>((half ? p.w_up : p.w_gate) + h0), (int64_t)p.hidden * 2, columns};
        const Matrix d = {reinterpret_cast<const char*>(p.d + (half * p.rows + r0) * p.inner), (int64_t)p.inner * 2, rows};
        typename P::LoadA la(w, wave * P::kLoadsA, p.inner, lane);
        typename P::LoadB lb(d, wave * P::kLoadsB, (int64_t)p.inner * 2, lane);
        c.add(la, lb, (p.inner + kStageRows - 1) / kStageRows, lds_address(lds), wave, lane);
    }
    int e = 0;
    if constexpr (F16)
        e = stored_exponent(p, slot);
    store<F16>(c, p.dx, r0 + 32 * P::first_b(wave), p.rows, h0 + 32 * P::first_a(wave), p.hidden, e, lane);
}

// Tiles of kRowsB rows (of one weight) and kRowsA columns of dw_gate and dw_up;
// the first half of the rows of tiles is dw_gate's.
template <bool F16, int N>
__global__ __launch_bounds__(256, N == 4 ? 1 : 2)
void feed_forward_dw_kernel(const BwdParams p)
{
    using P = Product<F16 ? kFp16 : kBf16, kColumns, kColumns, false, N, N, 2, 2>;
    __shared__ __attribute__((aligned(2 * P::kSlot))) char lds[P::kLds];
    __shared__ float slot[4];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const TileOf tile(blockIdx.x, p.row_tiles, p.column_tiles, 8);
    const int each = (int)p.row_tiles / 2, of_up = tile.row >= each;
    const int i0 = (tile.row - of_up * each) * P::kRowsB, h0 = tile.column * P::kRowsA;
    const int rows = p.inner - i0 < P::kRowsB ? p.inner - i0 : P::kRowsB;
    const int columns = p.hidden - h0 < P::kRowsA ? p.hidden - h0 : P::kRowsA;
    const Matrix x = {reinterpret_cast<const char*>(p.x + h0), (int64_t)p.hidden * 2, columns};
    const Matrix d = {reinterpret_cast<const char*>(p.d + of_up * p.rows * p.inner + i0), (int64_t)p.inner * 2, rows};
    P c;
    c.clear();
    typename P::LoadA la(x, wave * P::kLoadsA, p.rows, lane);
    typename P::LoadB lb(d, wave * P::kLoadsB, p.rows, lane);
    c.add(la, lb, (int)((p.rows + kStageRows - 1) / kStageRows), lds_address(lds), wave, lane);
    int e = 0;
    if constexpr (F16)
        e = p.rows ? stored_exponent(p, slot) : 0;
    uint16_t* out = of_up ? p.dw_up : p.dw_gate;
    store<F16>(c, out, i0 + 32 * P::first_b(wave), p.inner, h0 + 32 * P::first_a(wave), p.hidden, e, lane);
}

// ---------------------------------------------------------------- launches

using Fn = void (*)(BwdParams);

template <int ACT>
Fn select_gradients(bool f16)
{
    return f16 ? feed_forward_gradients_kernel<true, ACT> : feed_forward_gradients_kernel<false, ACT>;
}

Fn select_dx(bool f16, bool large)
{
    if (large)
        return f16 ? feed_forward_dx_kernel<true, 4> : feed_forward_dx_kernel<false, 4>;
    return f16 ? feed_forward_dx_kernel<true, 2> : feed_forward_dx_kernel<false, 2>;
}

Fn select_dw(bool f16, bool large)
{
    if (large)
        return f16 ? feed_forward_dw_kernel<true, 4> : feed_forward_dw_kernel<false, 4>;
    return f16 ? feed_forward_dw_kernel<true, 2> : feed_forward_dw_kernel<false, 2>;
}

// Workgroups of the elementwise passes: 16 KB of each tensor and more a workgroup,
// as many as keep the memory busy.
int64_t element_blocks(int64_t elements)
{
    const int64_t n = (elements + 4 * kThreads * kVec - 1) / (4 * kThreads * kVec);
    return n < 1 ? 1 : n > 2048 ? 2048 : n;
}

// Bytes of the workspace up to the array of the largest values.
int64_t largest_at(const dit_ff_args& a) { return 4 * a.rows * a.inner; }

}  // namespace

extern "C" int64_t dit_gated_feed_forward_backward_workspace_size(const dit_ff_args* args)
{
    const int rc = qkr_ff_host::check_args(args, false);
    if (rc != QKR_OK || args->rows == 0)
        return rc;
    const int64_t blocks = args->dtype == QKR_FP16 ? element_blocks(args->rows * args->inner) : 0;
    return largest_at(*args) + (blocks * 4 + 15) / 16 * 16;
}

extern "C" int dit_gated_feed_forward_backward(const dit_ff_args* args, const void* dh, const void* x,
                                               const void* w_gate, const void* w_up, const void* gate,
                                               const void* up, void* dx, void* dw_gate, void* dw_up,
                                               void* workspace, int64_t workspace_bytes, void* stream)
{
    using namespace qkr_ff_host;
    int rc = check_args(args, false);
    if (rc != QKR_OK)
        return rc;
    const dit_ff_args& a = *args;
    if (!dw_gate != !dw_up)
        return QKR_ERR_NULL;
    if ((!dx || a.rows == 0) && !dw_gate)
        return QKR_OK;
    if (a.rows && (!dh || !x || !gate || !up || (dx && (!w_gate || !w_up))))
        return QKR_ERR_NULL;
    const int64_t need = dit_gated_feed_forward_backward_workspace_size(args);
    if (need && (!workspace || workspace_bytes < need))
        return QKR_ERR_WORKSPACE;
    const uint64_t hidden = a.hidden, inner = a.inner, rows = a.rows;
    const uint64_t by_h = rows * hidden * 2, by_i = rows * inner * 2, by_w = inner * hidden * 2;
    const Buffer in[] = {{dh, by_i, 16}, {x, by_h, 16}, {gate, by_i, 16}, {up, by_i, 16},
                         {dx ? w_gate : nullptr, dx ? by_w : 0, 16}, {dx ? w_up : nullptr, dx ? by_w : 0, 16}};
    const Buffer out[] = {{dx, dx ? by_h : 0, 16}, {dw_gate, dw_gate ? by_w : 0, 16}, {dw_up, dw_up ? by_w : 0, 16},
                          {workspace, (uint64_t)need, 16}};
    if ((rc = check_buffers(in, 6, out, 4)) != QKR_OK)
        return rc;

    BwdParams p = {};
    p.dh = static_cast<const uint16_t*>(dh);
    p.x = static_cast<const uint16_t*>(x);
    p.w_gate = static_cast<const uint16_t*>(w_gate);
    p.w_up = static_cast<const uint16_t*>(w_up);
    p.gate = static_cast<const uint16_t*>(gate);
    p.up = static_cast<const uint16_t*>(up);
    p.dx = static_cast<uint16_t*>(dx);
    p.dw_gate = static_cast<uint16_t*>(dw_gate);
    p.dw_up = static_cast<uint16_t*>(dw_up);
    p.d = static_cast<uint16_t*>(workspace);
    p.largest = reinterpret_cast<float*>(static_cast<char*>(workspace) + largest_at(a));
    p.rows = a.rows;
    p.hidden = a.hidden;
    p.inner = a.inner;
    const bool f16 = a.dtype == QKR_FP16, silu = a.activation == DIT_FF_SILU;
    if (a.rows) {
        const int64_t blocks = element_blocks(a.rows * a.inner);
        p.largest_blocks = f16 ? (uint32_t)blocks : 0;
        if (f16)
            rc = launch(silu ? feed_forward_largest_kernel<0> : feed_forward_largest_kernel<1>, blocks, p, stream);
        if (rc == QKR_OK)
            rc = launch(silu ? select_gradients<0>(f16) : select_gradients<1>(f16), blocks, p, stream);
    }
    if (rc == QKR_OK && dx && a.rows) {
        const bool large = large_tiles(a.rows, a.hidden);
        const int64_t side = large ? 256 : 128;
        p.row_tiles = (uint32_t)((a.rows + side - 1) / side);
        p.column_tiles = (uint32_t)((a.hidden + side - 1) / side);
        rc = launch(select_dx(f16, large), (int64_t)p.row_tiles * p.column_tiles, p, stream);
    }
    if (rc == QKR_OK && dw_gate) {
        const bool large = large_tiles(2 * (int64_t)a.inner, a.hidden);
        const int64_t side = large ? 256 : 128;
        p.row_tiles = (uint32_t)(2 * ((a.inner + side - 1) / side));
        p.column_tiles = (uint32_t)((a.hidden + side - 1) / side);
        rc = launch(select_dw(f16, large), (int64_t)p.row_tiles * p.column_tiles, p, stream);
    }
    return rc;
}
