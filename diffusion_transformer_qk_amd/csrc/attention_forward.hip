// attention_forward.hip -- attention forward for gfx950 (see dit_attention.h).
//
// One wave holds 32 query rows as the B operand of S^T = K Q^T: its lane n has
// row n (twice, for the two halves of the wave), so the running maximum m and
// sum l of a row are plain registers and need one cross-lane step a tile.  The
// scores of a tile come out of the product with keys down the registers, which
// is the layout in which the packed probabilities are the B operand of
// O^T = V^T P^T (attention_common.h); P never goes through LDS.
//
// Query heads that share a key head are taken as rows of one sequence (row r
// is query r / G, head r % G of the group), so their K and V are staged once.
//
// K and V tiles are staged straight into a double buffer in LDS; the loads of
// tile t+1 run while tile t is computed.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "attention_common.h"
#include "attention_host.h"
#include "dit_attention.h"

namespace {

using namespace qkr_attn;

struct FwdParams {
    const uint16_t *q, *k, *v;
    uint16_t* out;
    float* lse;
    const int32_t* kv_lengths;
    int64_t q_bs, q_ts, q_hs, k_bs, k_ts, k_hs, v_bs, v_ts, v_hs, o_bs, o_ts, o_hs;
    int32_t q_tokens, kv_tokens, kv_heads, group, rows;    // rows = q_tokens * group
    int32_t row_blocks;
    uint32_t pairs;                           // batch * kv_heads
    int32_t splits;                           // of the key tiles
    float c;                                  // scale * log2(e)
    float* part_o;                            // [splits][batch * kv_heads * rows][D]
    float* part_lse;                          // [splits][batch * kv_heads * rows], base 2
};

// exp2 of the scores is taken relative to 2^-p_shift of the row's maximum, so
// that fp16 probabilities down to 2^-21 of the largest are normal numbers; a
// maximum is kept until the scores pass it by kSlack, so p <= 2^(p_shift + kSlack).
template <bool F16>
constexpr float p_shift() { return F16 ? 7.0f : 0.0f; }
constexpr float kSlack = 8.0f;

// Waves a SIMD that the registers have to allow (of 4-wave workgroups): q and
// o take 48, 96 or 192 of them a lane beside the scores (32 at head_dim 64, 16
// above) and the operands.
constexpr int waves_per_simd(int d) { return d == 64 ? 4 : d == 128 ? 3 : 2; }

// Keys of a tile.  head_dim 128: 64 keys, which leave two waves a SIMD, measured
// 1 to 2% slower on 32768 queries and 10% on 512 keys, where the last tile and the
// start of a workgroup count.  head_dim 64, where a tile's fixed work weighs most
// and the waves stay four: 32 heads of 4096 take 158 us with 64 keys, 168 with 32.
constexpr int tile_keys(int d, int waves) { return d == 64 && waves == 4 ? 64 : 32; }

template <int D, bool F16, bool CAUSAL, int NW>
__global__ __launch_bounds__(NW * 64, NW == 4 ? waves_per_simd(D) : D == 256 ? 1 : 2)
void attention_forward_kernel(const FwdParams p)
{
    constexpr int BM = NW * 32, BN = tile_keys(D, NW), KB = BN / 32, DB = D / 32;
    constexpr int kTile = BN * D * 2;
    // With one wave the call waits for memory, and p can have a second term,
    // what its rounding to 16 bits left: out is then off by its own rounding
    // alone.
    constexpr bool kTwoTerms = NW == 1;
    __shared__ __attribute__((aligned(4 * kTile))) char lds[4 * kTile];   // [buffer][K, V]
    const int lane = threadIdx.x % 64, n = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    const BlockOf block(blockIdx.x, p.pairs, p.row_blocks * p.splits);
    const int mb_raw = block.part % p.row_blocks, split = block.part / p.row_blocks;
    const uint32_t bh = block.pair;                      // sample, key head
    const int64_t b = bh / (uint32_t)p.kv_heads;
    const int hk = bh % (uint32_t)p.kv_heads;
    const int mb = CAUSAL ? p.row_blocks - 1 - mb_raw : mb_raw;   // the longest first

    int len = p.kv_tokens;
    if (p.kv_lengths) {
        const int given = __builtin_amdgcn_readfirstlane(p.kv_lengths[b]);
        len = given < 0 ? 0 : given < len ? given : len;
    }
    const int r0 = mb * BM + wave * 32;
    const int r = r0 + n < p.rows ? r0 + n : p.rows - 1;          // this lane's row
    const int qi = r / p.group, head = hk * p.group + r % p.group;
    const int shift = p.kv_tokens - p.q_tokens;                   // causal: sees keys <= qi + shift
    int end = len;                                                // keys of the workgroup
    if (CAUSAL) {
        const int last = (mb * BM + BM < p.rows ? mb * BM + BM : p.rows) - 1;
        const int sees = last / p.group + shift + 1;
        end = sees < end ? (sees < 0 ? 0 : sees) : end;
    }
    const int tiles = (end + BN - 1) / BN;
    // an even share of the tiles that this row block's masks leave
    const int each = (tiles + p.splits - 1) / p.splits;
    const int t0 = split * each, t1 = tiles < t0 + each ? tiles : t0 + each;
    // keys below this are seen by every row of the wave
    int open = len;
    if (CAUSAL) {
        const int s = (r0 < p.rows ? r0 : p.rows - 1) / p.group + shift + 1;
        open = s < open ? s : open;
    }

    u32x4 qf[D / 16];
    {
        const uint16_t* row = p.q + b * p.q_bs + qi * p.q_ts + head * p.q_hs + 8 * g;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            qf[kk] = load16<false>(row + 16 * kk);
    }
    f32x16 o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i)
        o[i] = f32x16{};
    float m = -INFINITY, l = 0.0f;         // m in units of log2 (scores times c)

    const Stager<D> ks(lane, p.k_ts), vs(lane, p.v_ts);
    const uint16_t* kbase = p.k + b * p.k_bs + hk * p.k_hs;
    const uint16_t* vbase = p.v + b * p.v_bs + hk * p.v_hs;
    uint32_t fill = lds_address(lds);
    TileAt at(fill, lane);
    const auto stage = [&](int t) {
        const int64_t first = (int64_t)t * BN;
        const int left = len - (int)first;
        if constexpr (NW == 4) {           // groups of 16 rows: two waves K's, two V's
#pragma unroll
            for (int i = 0; i < BN / 32; ++i) {
                if (wave < 2)
                    ks.load(kbase + first * p.k_ts, p.k_ts, left, fill, wave + 2 * i);
                else
                    vs.load(vbase + first * p.v_ts, p.v_ts, left, fill + kTile, wave - 2 + 2 * i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ks.load(kbase + first * p.k_ts, p.k_ts, left, fill, i);
                vs.load(vbase + first * p.v_ts, p.v_ts, left, fill + kTile, i);
            }
        }
        fill ^= 2 * kTile;
    };
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        settle(qf[kk]);

    if (t0 < t1)
        stage(t0);
    for (int t = t0; t < t1; ++t) {
        wait_staged();
        __syncthreads();       // tile t is there, and the other buffer is free
        if (t + 1 < t1)
            stage(t + 1);

        f32x16 s[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            s[j] = f32x16{};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                s[j] = mfma<F16>(row_fragment(at, j * block_bytes<D>(), kk), qf[kk], s[j]);
        }
        if (__builtin_expect(t * BN + BN > open, 0)) {          // some key of the tile is hidden from some row
            keep_branch();
            const int sees = CAUSAL ? (qi + shift + 1 < len ? qi + shift + 1 : len) : len;
#pragma unroll
            for (int j = 0; j < KB; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (t * BN + j * 32 + 8 * (i / 4) + 4 * g + i % 4 >= sees)
                        s[j][i] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                top = fmaxf(top, s[j][i]);
        top = half_max(top) * p.c;
        if (__builtin_expect(__any(top > m + kSlack) != 0, 0)) {
            const float m_new = fmaxf(m, top);
            const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - m_new);
            m = m_new;
            l *= f;
#pragma unroll
            for (int i = 0; i < DB; ++i)
                o[i] *= f;
        }
        // rows that have seen no key yet: every score is -inf, and p is 0
        const float base = (m == -INFINITY ? 0.0f : m) - p_shift<F16>();
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i], p.c, -base));
                sum += s[j][i];
            }
        l += sum;
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const u32x4 pf = pack_b<F16>(s[j], k);
                u32x4 rest;
                if constexpr (kTwoTerms)
                    rest = pack_rest<F16>(s[j], k, pf);
#pragma unroll
                for (int i = 0; i < DB; ++i) {
                    const u32x4 vf = tr_fragment(at, kTile + j * block_bytes<D>(), k, i);
                    o[i] = mfma<F16>(vf, pf, o[i]);
                    if constexpr (kTwoTerms)
                        o[i] = mfma<F16>(vf, rest, o[i]);
                }
            }
        at.flip(2 * kTile);
    }

    l = half_sum(l);
    const bool valid = r0 + n < p.rows;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float lse2 = l == 0.0f ? -INFINITY : m - p_shift<F16>() + __builtin_amdgcn_logf(l);
    if (p.splits == 1) {
        uint16_t* row = p.out + b * p.o_bs + qi * p.o_ts + head * p.o_hs;
#pragma unroll
        for (int i = 0; i < DB; ++i)
            store_column<F16>(row + 32 * i, o[i], inv, g, valid);
        if (valid && g == 0)
            p.lse[(b * p.kv_heads * p.group + head) * p.q_tokens + qi] = lse2 * kLn2;
    } else {
        const int64_t slot = (split * (int64_t)p.pairs + bh) * p.rows + r;
#pragma unroll
        for (int i = 0; i < DB; ++i)
            store_column_f32(p.part_o + slot * D + 32 * i, o[i], inv, g, valid);
        if (valid && g == 0)
            p.part_lse[slot] = lse2;
    }
}

// A row of out and its lse (given in base 2).
template <bool F16>
__device__ __forceinline__ void store_joined(const FwdParams& p, int64_t at, int col, f32x4 o, float lse2)
{
    const int64_t bh = at / p.rows, b = bh / p.kv_heads;
    const int r = at % p.rows, qi = r / p.group;
    const int head = (int)(bh % p.kv_heads) * p.group + r % p.group;
    *reinterpret_cast<u32x2*>(p.out + b * p.o_bs + qi * p.o_ts + head * p.o_hs + col) =
        u32x2{pack2<F16>(o[0], o[1]), pack2<F16>(o[2], o[3])};
    if (col == 0)
        p.lse[(b * p.kv_heads * p.group + head) * p.q_tokens + qi] = lse2 * kLn2;
}

// Joins the splits of a row: out = sum_k 2^(lse_k - lse) out_k.  D / 4 threads
// hold 4 columns each.  With many splits (kManySplits or more) a workgroup
// takes one row and its 1024 / D such sets every (1024 / D)th split; with fewer
// each set takes a row of its own.
constexpr int kManySplits = 16;

template <int D, bool F16, bool MANY>
__global__ __launch_bounds__(256)
void attention_join_kernel(const FwdParams p)
{
    constexpr int L = D / 4, S = 256 / L;
    const int set = threadIdx.x / L, col = threadIdx.x % L * 4;
    const int64_t total = (int64_t)p.pairs * p.rows;
    const int64_t at = MANY ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * S + set;
    float top = -INFINITY, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (MANY) {
        __shared__ float tops[4];
        for (int k = threadIdx.x; k < p.splits; k += 256)
            top = fmaxf(top, p.part_lse[k * total + at]);
        top = block_max<4>(top, tops);
    } else {
        if (at >= total)
            return;
        for (int k = 0; k < p.splits; ++k)
            top = fmaxf(top, p.part_lse[k * total + at]);
    }
    const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
    for (int k = MANY ? set : 0; k < p.splits; k += MANY ? S : 1) {
        const float w = __builtin_amdgcn_exp2f(p.part_lse[k * total + at] - base);
        l += w;
        o += w * *reinterpret_cast<const f32x4*>(p.part_o + (k * total + at) * D + col);
    }
    if constexpr (MANY) {
        __shared__ f32x4 sums[S][L];
        __shared__ float weights[S];
        sums[set][threadIdx.x % L] = o;
        if (threadIdx.x % L == 0)
            weights[set] = l;
        __syncthreads();
        if (set > 0)
            return;
#pragma unroll
        for (int i = 1; i < S; ++i) {
            o += sums[i][threadIdx.x];
            l += weights[i];
        }
    }
    o *= l == 0.0f ? 0.0f : 1.0f / l;
    store_joined<F16>(p, at, col, o, l == 0.0f ? -INFINITY : base + __builtin_amdgcn_logf(l));
}

struct Shape {
    int waves;
    int64_t row_blocks, splits;
};

// Up to 32 rows of a pair (one query, and a few) are one wave's: nothing is
// shared in the workgroup, and as many of them as their LDS allows keep loads
// in flight.  Calls that leave CUs idle cut the keys: into as many runs as fill
// the chip once, of at least 512 keys (128 for one wave, which waits for memory),
// or the launch that joins them costs what they save.
Shape shape_of(const dit_attn_args& a)
{
    Shape s;
    const int64_t rows = a.q_tokens * (a.heads / a.kv_heads);
    s.waves = rows <= 32 ? 1 : 4;
    s.row_blocks = (rows + 32 * s.waves - 1) / (32 * s.waves);
    const int64_t blocks = s.row_blocks * a.batch * a.kv_heads;
    const int keys = tile_keys(a.head_dim, s.waves);
    const int64_t tiles = (a.kv_tokens + keys - 1) / keys;
    // workgroups resident at once: four waves by their registers, one by the
    // double buffers in 160 KB of LDS a CU (8 at most, the waves of two SIMDs)
    const int64_t by_lds = 160 * 1024 / (8 * keys * a.head_dim);
    const int64_t resident = 256 * (s.waves == 4 ? waves_per_simd(a.head_dim) : by_lds > 8 ? 8 : by_lds);
    const int64_t least = (s.waves == 1 ? 128 : 512) / keys;
    s.splits = 1;
    if (blocks > 0 && 2 * blocks <= resident && tiles >= 2 * least) {
        s.splits = resident / blocks;
        if (s.splits > tiles / least)
            s.splits = tiles / least;
    }
    return s;
}

using Fn = void (*)(FwdParams);

template <int D, bool F16, bool CAUSAL>
Fn select(int waves)
{
    return waves == 1 ? attention_forward_kernel<D, F16, CAUSAL, 1>
                      : attention_forward_kernel<D, F16, CAUSAL, 4>;
}

template <int D>
Fn select(bool f16, bool causal, int waves)
{
    if (f16)
        return causal ? select<D, true, true>(waves) : select<D, true, false>(waves);
    return causal ? select<D, false, true>(waves) : select<D, false, false>(waves);
}

template <int D>
Fn select_join(bool f16, bool many)
{
    if (many)
        return f16 ? attention_join_kernel<D, true, true> : attention_join_kernel<D, false, true>;
    return f16 ? attention_join_kernel<D, true, false> : attention_join_kernel<D, false, false>;
}

}  // namespace

extern "C" int64_t dit_attention_workspace_size(const dit_attn_args* args)
{
    const int rc = qkr_attn_host::check_args(args);
    if (rc != QKR_OK)
        return rc;
    const Shape s = shape_of(*args);
    if (s.splits == 1)
        return 0;
    return s.splits * args->batch * args->heads * args->q_tokens * (args->head_dim + 1) * 4;
}

extern "C" int dit_attention(const dit_attn_args* args, const dit_attn_tensor* q,
                             const dit_attn_tensor* k, const dit_attn_tensor* v,
                             const dit_attn_tensor* out, float* lse, void* workspace,
                             int64_t workspace_bytes, void* stream)
{
    using namespace qkr_attn_host;
    int rc = check_args(args);
    if (rc != QKR_OK)
        return rc;
    const dit_attn_args& a = *args;
    if (a.batch == 0 || a.q_tokens == 0)
        return QKR_OK;
    const Extent eq = {a.q_tokens, a.heads}, ekv = {a.kv_tokens, a.kv_heads};
    const dit_attn_tensor tq = plain(a, q, eq), tk = plain(a, k, ekv), tv = plain(a, v, ekv),
                          to = plain(a, out, eq);
    if ((rc = check_tensor(a, tq, eq, false)) || (rc = check_tensor(a, tk, ekv, false)) ||
        (rc = check_tensor(a, tv, ekv, false)) || (rc = check_tensor(a, to, eq, true)))
        return rc;
    const uint64_t lse_bytes = (uint64_t)a.batch * a.heads * a.q_tokens * 4;
    if (!lse)
        return QKR_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(lse) & 3u || reinterpret_cast<uintptr_t>(a.kv_lengths) & 3u)
        return QKR_ERR_ALIGN;
    const int64_t need = dit_attention_workspace_size(args);
    if (need && (!workspace || workspace_bytes < need))
        return QKR_ERR_WORKSPACE;
    if (!qkr_host::aligned16(workspace))
        return QKR_ERR_ALIGN;
    const Range lse_r = {lse, lse_bytes}, ws_r = {workspace, (uint64_t)need};
    const Range len_r = {a.kv_lengths, a.kv_lengths ? (uint64_t)a.batch * 4 : 0};
    const Range in[] = {range(a, tq, eq), range(a, tk, ekv), range(a, tv, ekv), len_r};
    const Range o = range(a, to, eq);
    for (const Range& x : in)
        if (meet(x, lse_r) || meet(x, ws_r))
            return QKR_ERR_ARG;
    if (meet(o, lse_r) || meet(o, ws_r) || meet(lse_r, ws_r) || meet(o, len_r) ||
        may_meet(a, to, eq, tq, eq) || may_meet(a, to, eq, tk, ekv) || may_meet(a, to, eq, tv, ekv))
        return QKR_ERR_ARG;

    const Shape s = shape_of(a);
    FwdParams p = {};
    unpack(tq, p.q, p.q_bs, p.q_ts, p.q_hs);
    unpack(tk, p.k, p.k_bs, p.k_ts, p.k_hs);
    unpack(tv, p.v, p.v_bs, p.v_ts, p.v_hs);
    unpack(to, p.out, p.o_bs, p.o_ts, p.o_hs);
    p.lse = lse;
    p.kv_lengths = a.kv_lengths;
    p.q_tokens = (int32_t)a.q_tokens;
    p.kv_tokens = (int32_t)a.kv_tokens;
    p.kv_heads = a.kv_heads;
    p.group = a.heads / a.kv_heads;
    p.rows = (int32_t)(a.q_tokens * p.group);
    p.row_blocks = (int32_t)s.row_blocks;
    p.pairs = (uint32_t)(a.batch * a.kv_heads);
    p.splits = (int32_t)s.splits;
    p.c = a.scale * kLog2e;
    const int64_t total = a.batch * a.kv_heads * (int64_t)p.rows;
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = p.part_o ? p.part_o + s.splits * total * a.head_dim : nullptr;
    const bool f16 = a.dtype == QKR_FP16, causal = a.causal != 0;
    Fn fn = a.head_dim == 64    ? select<64>(f16, causal, s.waves)
            : a.head_dim == 128 ? select<128>(f16, causal, s.waves)
                                : select<256>(f16, causal, s.waves);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    void* argv[] = {&p};
    hipError_t err = hipLaunchKernel(reinterpret_cast<const void*>(fn),
                                     dim3((unsigned)(p.pairs * s.splits * s.row_blocks)),
                                     dim3(s.waves * 64), argv, 0, st);
    if (err == hipSuccess && s.splits > 1) {
        const bool many = s.splits >= kManySplits;
        fn = a.head_dim == 64    ? select_join<64>(f16, many)
             : a.head_dim == 128 ? select_join<128>(f16, many)
                                 : select_join<256>(f16, many);
        const int64_t rows = many ? 1 : 1024 / a.head_dim;
        err = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)((total + rows - 1) / rows)),
                              dim3(256), argv, 0, st);
    }
    return err == hipSuccess ? QKR_OK : QKR_ERR_HIP;
}
