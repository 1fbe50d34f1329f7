// gated_feed_forward_backward.hip -- dx, dw_gate and dw_up for gfx950 (see
// feed_forward.h).
//
// First dgate and dup, element by element from dh, gate and up, into the
// workspace; then two products (feed_forward_common.h), each of both halves at
// once:
//   dx = dgate W_gate + dup W_up: one sum over 2 * inner, the weights read down
//        their rows by transposed reads of LDS;
//   dw = dgate^T x and dup^T x: sums over the rows, both operands read down.
// 4608 rows of 6144 and 16384 columns: 122 us, 1.53 ms (1215 TFLOP/s) and 1.40 (1326;
// the library's products 2.05 and 1.61).  The first pass moves 755 MB at 6.2 TB/s.
//
// Calls of few rows or numbers (terms_of) round dgate and dup in two terms: the
// remainders are rows beside theirs, so that the weights are read once for both.
//
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
    uint16_t* d;              // [2][terms][rows][inner]: dgate and dup, each with what its rounding left, if terms is 2
    int32_t terms;
    uint16_t* x_twice;        // [2][rows][hidden]: x beside itself for the terms' rows in dw, or NULL
    float* largest;           // fp16: [largest_blocks] largest finite |dgate|, |dup|
    uint32_t largest_blocks;
    int64_t rows;
    int32_t hidden, inner;
    uint32_t row_tiles, column_tiles;   // of the grid
    int32_t splits;           // of k
    float* parts;             // [splits][terms][rows][hidden] of dx, or [splits][2 inner][hidden] of dw, or NULL where
                              // the products themselves store dx or dw
};

constexpr int kThreads = 256;

// The power of two that dgate and dup are divided by: the largest becomes 2^14 .. 2^15.
template <int THREADS>
__device__ __forceinline__ int stored_exponent(const BwdParams& p, float* slot)
{
    float top = 0.0f;
    for (uint32_t i = threadIdx.x; i < p.largest_blocks; i += THREADS)
        top = fmaxf(top, p.largest[i]);
    top = block_max<THREADS / 64>(top, slot);
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

// What rounding v to `rounded` left (nothing of an infinity or NaN).
template <bool F16>
__device__ __forceinline__ u32x4 rest8(const float (&v)[8], u32x4 rounded)
{
    float r[8];
    unpack8<F16>(rounded, r);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        r[k] = fabsf(r[k]) <= 0x1.fffffep127f ? v[k] - r[k] : 0.0f;
    return pack8<F16>(r);
}

template <bool F16, int ACT>
__global__ __launch_bounds__(kThreads)
void feed_forward_gradients_kernel(const BwdParams p)
{
    __shared__ float slot[4];
    const int64_t n = p.rows * p.inner;
    int e = 0;
    if constexpr (F16)
        e = stored_exponent<kThreads>(p, slot);
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
        const u32x4 da = pack8<F16>(a), db = pack8<F16>(b);
        uint16_t* up = p.d + p.terms * n;
        store16<false>(p.d + i, da);
        store16<false>(up + i, db);
        if (p.terms == 2) {
            store16<false>(p.d + n + i, rest8<F16>(a, da));
            store16<false>(up + n + i, rest8<F16>(b, db));
        }
    }
    if (!p.x_twice)
        return;
    const int64_t of_x = p.rows * p.hidden;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kVec; i < of_x;
         i += (int64_t)gridDim.x * kThreads * kVec) {
        const u32x4 x = load16<false>(p.x + i);
        store16<false>(p.x_twice + i, x);
        store16<false>(p.x_twice + of_x + i, x);
    }
}

// A wave's sums to rows from r0 on (of `rows`) and columns from a0 on of [rows,
// columns]: times 2^e to `out`, or as they are to a split's part.
template <bool F16, typename P>
__device__ __forceinline__ void store(P& c, uint16_t* out, float* part, int64_t r0, int64_t rows, int a0,
                                      int columns, int e, int lane)
{
    constexpr int kBlocks = P::kTilesA * P::kSide / 32;
    unrolled<P::kPieces * kBlocks>([&](auto number) __attribute__((always_inline)) {
        constexpr int q = decltype(number)::value / kBlocks, i = decltype(number)::value % kBlocks;
        const int64_t r = r0 + P::piece_row(q, lane);
        float v[8];
        c.template piece<i, q>(v);
        const int a = a0 + 32 * i;
        if (part) {
#pragma unroll
            for (int run = 0; run < 2; ++run) {
                const int at = a + P::piece_column(q, lane, run);
                if (r < rows && at < columns)
                    *reinterpret_cast<f32x4*>(part + r * columns + at) =
                        f32x4{v[4 * run], v[4 * run + 1], v[4 * run + 2], v[4 * run + 3]};
            }
            return;
        }
        if constexpr (F16) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = __builtin_amdgcn_ldexpf(v[k], e);
        }
        P::template store_piece<F16>(out + r * columns + a, v, q, lane, r < rows, columns - a);
    });
}

// Tiles of kRowsB rows and kRowsA columns of dx, whose terms are rows beside each other
// here: the weights are read once for both, and the parts are added by the join.
template <bool F16, int N>
__global__ __launch_bounds__(128 * N, 2)
void feed_forward_dx_kernel(const BwdParams p)
{
    using P = Product<F16 ? kFp16 : kBf16, kColumns, kRows, false, N, 2, 2, N>;
    __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t tiles = p.row_tiles * p.column_tiles;
    const TileOf tile(blockIdx.x % tiles, p.row_tiles, p.column_tiles, 4);
    const int split = blockIdx.x / tiles;
    const int64_t all_rows = p.terms * p.rows, r0 = (int64_t)tile.row * P::kRowsB, rows_left = all_rows - r0;
    const int h0 = tile.column * P::kRowsA;
    const int rows = rows_left < P::kRowsB ? (int)rows_left : P::kRowsB;
    const int columns = p.hidden - h0 < P::kRowsA ? p.hidden - h0 : P::kRowsA;
    P c;
    c.clear();
    // the split's stages of both halves' together
    const int stages = (p.inner + kStageRows - 1) / kStageRows, each = (2 * stages + p.splits - 1) / p.splits;
    const int from = split * each, to = from + each < 2 * stages ? from + each : 2 * stages;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const int low = (from > half * stages ? from : half * stages) - half * stages;
        const int high = (to < (half + 1) * stages ? to : (half + 1) * stages) - half * stages;
        if (low >= high)
            continue;
        const int k0 = low * kStageRows, k = (high * kStageRows < p.inner ? high * kStageRows : p.inner) - k0;
        const Matrix w = {reinterpret_cast<const char*>((half ? p.w_up : p.w_gate) + (int64_t)k0 * p.hidden + h0),
                          (int64_t)p.hidden * 2, columns};
        const Matrix d = {reinterpret_cast<const char*>(p.d + (half * all_rows + r0) * p.inner + k0),
                          (int64_t)p.inner * 2, rows};
        typename P::LoadA la(w, wave * P::kLoadsA, k, lane);
        typename P::LoadB lb(d, wave * P::kLoadsB, (int64_t)k * 2, lane);
        c.add(la, lb, high - low, lds_address(lds), wave, lane);
    }
    int e = 0;
    if constexpr (F16)
        e = stored_exponent<64 * P::kWaves>(p, reinterpret_cast<float*>(lds));
    store<F16>(c, p.dx, p.parts ? p.parts + split * all_rows * p.hidden : nullptr, r0 + 32 * P::first_b(wave),
               all_rows, h0 + 32 * P::first_a(wave), p.hidden, e, lane);
}

// Tiles of kRowsB rows (of one weight) and kRowsA columns of dw_gate and dw_up;
// the first half of the rows of tiles is dw_gate's.  The sum runs over the rows of all
// terms.
template <bool F16, int N>
__global__ __launch_bounds__(128 * N, 2)
void feed_forward_dw_kernel(const BwdParams p)
{
    using P = Product<F16 ? kFp16 : kBf16, kColumns, kColumns, false, N, 2, 2, N>;
    __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t tiles = p.row_tiles * p.column_tiles;
    const TileOf tile(blockIdx.x % tiles, p.row_tiles, p.column_tiles, 4);
    const int split = blockIdx.x / tiles;
    const int per_weight = (int)p.row_tiles / 2, of_up = tile.row >= per_weight;
    const int i0 = (tile.row - of_up * per_weight) * P::kRowsB, h0 = tile.column * P::kRowsA;
    const int rows = p.inner - i0 < P::kRowsB ? p.inner - i0 : P::kRowsB;
    const int columns = p.hidden - h0 < P::kRowsA ? p.hidden - h0 : P::kRowsA;
    const int64_t all_rows = p.terms * p.rows;
    const int64_t stages = (all_rows + kStageRows - 1) / kStageRows, each = (stages + p.splits - 1) / p.splits;
    const int64_t low = split * each, high = low + each < stages ? low + each : stages;
    const int64_t k0 = low * kStageRows, k = (high * kStageRows < all_rows ? high * kStageRows : all_rows) - k0;
    P c;
    c.clear();
    if (low < high) {
        const Matrix x = {reinterpret_cast<const char*>((p.x_twice ? p.x_twice : p.x) + k0 * p.hidden + h0),
                          (int64_t)p.hidden * 2, columns};
        const Matrix d = {reinterpret_cast<const char*>(p.d + (of_up * all_rows + k0) * p.inner + i0),
                          (int64_t)p.inner * 2, rows};
        typename P::LoadA la(x, wave * P::kLoadsA, k, lane);
        typename P::LoadB lb(d, wave * P::kLoadsB, k, lane);
        c.add(la, lb, (int)(high - low), lds_address(lds), wave, lane);
    }
    int e = 0;
    if constexpr (F16)
        e = p.rows ? stored_exponent<64 * P::kWaves>(p, reinterpret_cast<float*>(lds)) : 0;
    float* part = p.parts ? p.parts + ((int64_t)split * 2 + of_up) * p.inner * p.hidden : nullptr;
    store<F16>(c, of_up ? p.dw_up : p.dw_gate, part, i0 + 32 * P::first_b(wave), p.inner,
               h0 + 32 * P::first_a(wave), p.hidden, e, lane);
}

// Adds `splits` parts in order (the splits', and for dx each term's): `first` and
// `second` are the halves of what they are parts of (`elements` each; no second for dx).
template <bool F16>
__global__ __launch_bounds__(kThreads)
void feed_forward_join_kernel(const BwdParams p, uint16_t* first, uint16_t* second, int64_t elements)
{
    __shared__ float slot[4];
    int e = 0;
    if constexpr (F16)
        e = stored_exponent<kThreads>(p, slot);
    const int64_t total = second ? 2 * elements : elements;
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kVec;
    if (i >= total)
        return;
    float sum[8] = {};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        float v[8];
        load_f32x8(p.parts + s * total + i, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum[k] += v[k];
    }
    if constexpr (F16) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum[k] = __builtin_amdgcn_ldexpf(sum[k], e);
    }
    store16<false>(i < elements ? first + i : second + (i - elements), pack8<F16>(sum));
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

// How both products are cut, and where the workspace's parts begin (in bytes).
struct Shape {
    qkr_ff_host::Cut dx, dw;
    int64_t terms, blocks, x_twice, largest, parts, bytes;
};

Shape shape_of(const dit_ff_args& a)
{
    Shape s;
    s.terms = qkr_ff_host::terms_of(a);
    s.dx = qkr_ff_host::cut_of(s.terms * a.rows, a.hidden, 2 * (((int64_t)a.inner + kStageRows - 1) / kStageRows), true);
    s.dw = qkr_ff_host::cut_of(2 * (int64_t)a.inner, a.hidden, (s.terms * a.rows + kStageRows - 1) / kStageRows, true);
    // tiles of one weight each
    const int64_t side = s.dw.large ? 256 : 128;
    s.dw.row_tiles = 2 * ((a.inner + side - 1) / side);
    s.blocks = element_blocks(a.rows * (s.terms == 2 && a.hidden > a.inner ? a.hidden : a.inner));
    s.x_twice = 4 * s.terms * a.rows * a.inner;
    s.largest = s.x_twice + (s.terms == 2 ? 4 * a.rows * a.hidden : 0);
    s.parts = s.largest + (a.dtype == QKR_FP16 ? (s.blocks * 4 + 15) / 16 * 16 : 0);
    const int64_t dx_parts = s.dx.splits * s.terms, dx = dx_parts > 1 ? dx_parts * a.rows * a.hidden * 4 : 0;
    const int64_t dw = s.dw.splits > 1 ? s.dw.splits * 2 * a.inner * a.hidden * 4 : 0;
    s.bytes = a.rows == 0 ? 0 : s.parts + (dx > dw ? dx : dw);
    return s;
}

hipError_t join(BwdParams p, uint16_t* first, uint16_t* second, int64_t elements, bool f16, void* stream)
{
    void* argv[] = {&p, &first, &second, &elements};
    const int64_t total = second ? 2 * elements : elements, per = kThreads * kVec;
    const void* fn = f16 ? reinterpret_cast<const void*>(feed_forward_join_kernel<true>)
                         : reinterpret_cast<const void*>(feed_forward_join_kernel<false>);
    return hipLaunchKernel(fn, dim3((unsigned)((total + per - 1) / per)), dim3(kThreads), argv, 0,
                           static_cast<hipStream_t>(stream));
}

}  // namespace

extern "C" int64_t dit_gated_feed_forward_backward_workspace_size(const dit_ff_args* args)
{
    const int rc = qkr_ff_host::check_args(args, false);
    return rc != QKR_OK ? rc : shape_of(*args).bytes;
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
    const Shape shape = shape_of(a);
    const int64_t need = shape.bytes;
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
    p.terms = (int32_t)shape.terms;
    p.x_twice = dw_gate && a.rows && shape.terms == 2
                    ? reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + shape.x_twice) : nullptr;
    p.largest = reinterpret_cast<float*>(static_cast<char*>(workspace) + shape.largest);
    p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + shape.parts);
    p.rows = a.rows;
    p.hidden = a.hidden;
    p.inner = a.inner;
    const bool f16 = a.dtype == QKR_FP16, silu = a.activation == DIT_FF_SILU;
    if (a.rows) {
        const int64_t blocks = shape.blocks;
        p.largest_blocks = f16 ? (uint32_t)blocks : 0;
        if (f16)
            rc = launch(silu ? feed_forward_largest_kernel<0> : feed_forward_largest_kernel<1>, blocks, p, stream);
        if (rc == QKR_OK)
            rc = launch(silu ? select_gradients<0>(f16) : select_gradients<1>(f16), blocks, p, stream);
    }
    float* const parts = p.parts;
    // `count` parts of `elements` (first and second together) are to be added
    const auto product = [&](const Cut& cut, Fn fn, int64_t count, uint16_t* first, uint16_t* second, int64_t elements) {
        p.row_tiles = (uint32_t)cut.row_tiles;
        p.column_tiles = (uint32_t)cut.column_tiles;
        p.splits = (int32_t)cut.splits;
        p.parts = count > 1 ? parts : nullptr;
        rc = launch(fn, cut.row_tiles * cut.column_tiles * cut.splits, p, stream, cut.large ? 512 : 256);
        p.splits = (int32_t)count;
        if (rc == QKR_OK && count > 1 && join(p, first, second, elements, f16, stream) != hipSuccess)
            rc = QKR_ERR_HIP;
    };
    if (rc == QKR_OK && dx && a.rows)
        product(shape.dx, select_dx(f16, shape.dx.large), shape.dx.splits * shape.terms, p.dx, nullptr, a.rows * a.hidden);
    if (rc == QKR_OK && dw_gate)
        product(shape.dw, select_dw(f16, shape.dw.large), shape.dw.splits, p.dw_gate, p.dw_up,
                (int64_t)a.inner * a.hidden);
    return rc;
}
