// attention_backward.hip -- attention backward for gfx950 (see dit_attention.h).
//
// Two launches, the second in two parts:
//   rows: lse (in base 2; for fp16 less the power of two of p) and delta =
//         dout . out of every query, and for fp16 the norms that bound dout . v;
//   dkv:  a wave owns 32 keys, keeps their k, v, dk and dv in registers and
//         walks the queries: S = Q K^T and dP = dO V^T come out with queries
//         down the registers, so packed P and dS are the B operands of
//         dV^T = dO^T P and dK^T = Q^T dS as they stand;
//   dq:   a wave owns 32 query rows and walks the keys, with S^T = K Q^T,
//         dP^T = V dO^T and dQ^T = K^T dS^T.
// The scores are computed twice (7 products instead of 5), because the other
// way, one walk that adds to dQ from every key block, needs fp32 atomic
// additions: their order changes the result from run to run, and their
// traffic is Sk / (keys of a workgroup) times the size of dQ in fp32.
//
// fp16: p = exp(s - lse) is about 1 / keys, and ds that times the gradient's
// size; both would sink into fp16's subnormals.  p is computed times 2^15
// (p <= 1), and dp - delta, which the norms of dout and v bound, is brought
// below 1 by a power of two (of a query in dq; of a whole key head in dkv,
// where queries are summed); the sums are scaled back in fp32.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "attention_common.h"
#include "attention_host.h"
#include "dit_attention.h"

namespace {

using namespace qkr_attn;

struct BwdParams {
    const uint16_t *dout, *q, *k, *v, *out;
    const float* lse;
    uint16_t *dq, *dk, *dv;
    const int32_t* kv_lengths;
    int64_t do_bs, do_ts, do_hs, q_bs, q_ts, q_hs, k_bs, k_ts, k_hs, v_bs, v_ts, v_hs;
    int64_t o_bs, o_ts, o_hs, dq_bs, dq_ts, dq_hs, dk_bs, dk_ts, dk_hs, dv_bs, dv_ts, dv_hs;
    int64_t batch;
    uint32_t pairs;                           // batch * kv_heads
    int32_t q_tokens, kv_tokens, heads, kv_heads, group, rows;
    int32_t row_blocks, key_blocks;
    int32_t column_waves;                     // waves to a block of keys, in dkv (DS)
    int32_t row_splits;                       // of the query tiles, in dkv
    int32_t key_splits;                       // of the key tiles, in dq
    int32_t stat_blocks, value_blocks;        // runs of a head's rows, of a key head's values
    float scale, c;                           // c = scale * log2(e)
    float* stats;                             // [batch][heads][q_tokens][lse2, delta]
    float* row_norms;                         // fp16: [batch][heads][stat_blocks] largest |dout|
    float* value_norms;                       // fp16: [batch][kv_heads][value_blocks] largest |v|
    float* part_kv;                           // [row_splits][pairs][kv_tokens][dk, dv][D]
    float* part_q;                            // [key_splits][pairs][rows][D]
    Rows q_rows, kv_rows;                     // packed sequences (batch is 1, rows all of the buffer's)
    int32_t fill_rest;
};

// Block `block` of SIZE rows (times `group`) of packed sequences.
template <int SIZE>
struct PackedBlock {
    int seq, at;              // the sequence, and the block's place in it
    int q_at, kv_at;          // the sequence's first rows
    int q_tokens, kv_tokens;

    // `of`: q_rows or kv_rows, by which the blocks are numbered
    __device__ __forceinline__ PackedBlock(const BwdParams& p, const Rows& of, int group, int block)
    {
        seq = sequence_of<SIZE>(of, group, block);
        at = __builtin_amdgcn_readfirstlane(block - first_block<SIZE>(of, group, seq));
        const int q0 = p.q_rows.first(seq), k0 = p.kv_rows.first(seq);
        const int q = p.q_rows.first(seq + 1) - q0, k = p.kv_rows.first(seq + 1) - k0;
        q_at = __builtin_amdgcn_readfirstlane(q0);
        kv_at = __builtin_amdgcn_readfirstlane(k0);
        q_tokens = __builtin_amdgcn_readfirstlane(q < 0 ? 0 : q);
        kv_tokens = __builtin_amdgcn_readfirstlane(k < 0 ? 0 : k);
    }

    // Whether rows `rows` (of the sequence, times the group) begin before this block and
    // are anybody's.
    __device__ __forceinline__ bool there(const BwdParams& p, int rows) const
    {
        return at >= 0 && at < (rows + SIZE - 1) / SIZE && (p.fill_rest || !p.q_rows.rest(seq));
    }
};

template <bool F16>
constexpr float p_shift() { return F16 ? 15.0f : 0.0f; }

// Exponent e of a bound on |dp|: |dp - delta| * 2^(-e - 1) <= 1.
__device__ __forceinline__ int bound_exponent(float bound)
{
    // a bound that is 0, infinite or NaN scales nothing
    if (!(bound > 0.0f && bound <= 0x1.fffffep127f))
        return -1;
    return __builtin_amdgcn_frexp_expf(bound);
}

// A row's squared norm, or 0 if it holds an infinity or NaN: such a row is lost
// whatever scales it, and counted it would leave all others unscaled, those
// that causality hides from it among them.
__device__ __forceinline__ float finite(float sq) { return sq <= 0x1.fffffep127f ? sq : 0.0f; }

// Rows of a workgroup of the kernel below: 32 queries a wave, or D / 8 lanes a
// value, 4 values each.
constexpr int kStatRows = 128;
constexpr int value_rows(int d) { return 4 * 256 / (d / 8); }

// lse2 (above) and delta of a run of one head's queries.  fp16: also the
// largest |dout| of the run, and in further workgroups the largest |v| of a run
// of a key head's values in use.
//
// delta is the diagonal of out dout^T, taken on the matrix cores in the order
// in which dout . v is summed: where out is a copy of one value (a query that
// sees one key, or gives one all its weight) dp - delta is then exactly 0, and
// not what two orders of summation differ by.  The fragments that takes, 16 bytes
// of a row a lane, cost time: 28 us on 4608 tokens of 48 heads of 128, where whole
// rows summed side by side took 21 (22 at a copy's rate).
// Packed: blocks are numbered by the sequences, those that no sequence needs have
// no rows.
template <int D, bool F16, bool PACKED>
__global__ __launch_bounds__(256)
void row_stats_kernel(const BwdParams p)
{
    __shared__ float tops[4];
    const int64_t rows = p.batch * p.heads * p.stat_blocks;
    float top = 0.0f;
    if (blockIdx.x < rows) {
        const int lane = threadIdx.x % 64, n = lane & 31, g = lane >> 5;
        const int64_t bh = blockIdx.x / p.stat_blocks, b = bh / p.heads;
        const int h = bh % p.heads;
        int64_t qi = (int64_t)(blockIdx.x % p.stat_blocks) * kStatRows + threadIdx.x / 64 * 32 + n;
        bool there = qi < p.q_tokens;
        if constexpr (PACKED) {
            const PackedBlock<kStatRows> of(p, p.q_rows, 1, (int)(blockIdx.x % p.stat_blocks));
            qi = (int64_t)of.at * kStatRows + threadIdx.x / 64 * 32 + n;
            there = of.at >= 0 && qi < of.q_tokens && !p.q_rows.rest(of.seq);
            qi += of.q_at;
        }
        const uint16_t* dor = p.dout + b * p.do_bs + qi * p.do_ts + h * p.do_hs + 8 * g;
        const uint16_t* outr = p.out + b * p.o_bs + qi * p.o_ts + h * p.o_hs + 8 * g;
        u32x4 df[D / 16], of[D / 16];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            df[kk] = there ? load16<false>(dor + 16 * kk) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            of[kk] = there ? load16<false>(outr + 16 * kk) : u32x4{0, 0, 0, 0};
        f32x16 c{};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            c = mfma<F16>(of[kk], df[kk], c);
        float delta = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (8 * (i / 4) + 4 * g + i % 4 == n)
                delta = c[i];
        if (there && ((n >> 2) & 1) == g) {     // the half of the wave that holds row n of column n
            const float lse = p.lse[bh * p.q_tokens + qi];
            // a query without keys: exp2(s - inf) is 0 for every score
            const float lse2 = lse == -INFINITY ? INFINITY : __builtin_fmaf(lse, kLog2e, -p_shift<F16>());
            reinterpret_cast<f32x2*>(p.stats)[bh * p.q_tokens + qi] = f32x2{lse2, delta};
        }
        if constexpr (F16) {
            float sq = 0.0f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                float x[8];
                unpack8<true>(df[kk], x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sq = __builtin_fmaf(x[i], x[i], sq);
            }
            top = finite(half_sum(sq));
        }
    } else if constexpr (F16) {
        constexpr int L = D / 8, R = 256 / L;
        const int d0 = threadIdx.x % L * 8, row0 = threadIdx.x / L;
        const int64_t at = blockIdx.x - rows, bh = at / p.value_blocks, b = bh / p.kv_heads;
        int len = p.kv_tokens;
        if (p.kv_lengths && p.kv_lengths[b] < len)
            len = p.kv_lengths[b];
        const uint16_t* vr = p.v + b * p.v_bs + bh % p.kv_heads * p.v_hs + d0;
        int64_t first = at % p.value_blocks * value_rows(D);
        if constexpr (PACKED) {
            const PackedBlock<value_rows(D)> of(p, p.kv_rows, 1, (int)(at % p.value_blocks));
            first = of.at < 0 ? 0 : (int64_t)of.at * value_rows(D);
            len = of.at < 0 || p.q_rows.rest(of.seq) ? 0 : of.kv_tokens;
            vr += of.kv_at * p.v_ts;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t j = first + i * R + row0;
            float x[8], sq = 0.0f;
            unpack8<true>(j < len ? load16<false>(vr + j * p.v_ts) : u32x4{0, 0, 0, 0}, x);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sq = __builtin_fmaf(x[k], x[k], sq);
#pragma unroll
            for (int w = 1; w < L; w *= 2)
                sq += __shfl_xor(sq, w);
            top = fmaxf(top, finite(sq));
        }
    }
    if constexpr (F16) {
        top = block_max<4>(top, tops);
        if (threadIdx.x == 0)
            (blockIdx.x < rows ? p.row_norms : p.value_norms - rows)[blockIdx.x] = sqrtf(top);
    }
}

// The largest of n values, by all threads of a workgroup of 4 waves.
__device__ __forceinline__ float largest(const float* v, int n, float* slot)
{
    float top = 0.0f;
    for (int i = threadIdx.x; i < n; i += 256)
        top = fmaxf(top, v[i]);
    return block_max<4>(top, slot);
}

// The largest of what row_stats_kernel left of blocks of SIZE rows for a sequence
// of packed ones, of `heads` heads from `head` on (of `blocks` values each).
template <int SIZE>
__device__ __forceinline__ float largest_packed(const float* v, int64_t head, int heads, int blocks,
                                                const Rows& rows, int seq, int tokens, float* slot)
{
    const int first = first_block<SIZE>(rows, 1, seq), n = (tokens + SIZE - 1) / SIZE;
    float top = 0.0f;
    for (int h = 0; h < heads; ++h)
        for (int i = threadIdx.x; i < n; i += 256)
            top = fmaxf(top, v[(head + h) * blocks + first + i]);
    return block_max<4>(top, slot);
}

constexpr int kWaves = 4;
constexpr int kTileRows = 64;      // queries (dk and dv) or keys (dq) staged at a time

// What a workgroup computes.
struct Work {
    uint32_t bh;                           // sample, key head
    int split, block, seq;                 // of the tiles; of keys or rows, of the sample or sequence
    int q_tokens, kv_tokens, rows, len;    // of the sample or sequence; len: its keys that are there
    int64_t q_at, kv_at;                   // the sequence's first rows

    __device__ __forceinline__ Work(const BwdParams& p, uint32_t bh, int split, int block)
        : bh(bh), split(split), block(block), seq(0), q_tokens(p.q_tokens), kv_tokens(p.kv_tokens),
          rows(p.rows), len(p.kv_tokens), q_at(0), kv_at(0)
    {
    }

    // `of`: the block that is `block` of all sequences' together, and there()
    template <int SIZE>
    __device__ __forceinline__ void in_sequence(const BwdParams& p, const PackedBlock<SIZE>& of)
    {
        const bool rest = p.q_rows.rest(of.seq);
        seq = of.seq;
        block = of.at;
        q_at = of.q_at;
        kv_at = of.kv_at;
        q_tokens = of.q_tokens;
        kv_tokens = of.kv_tokens;
        rows = q_tokens * p.group;
        len = rest ? 0 : kv_tokens;
    }

    __device__ __forceinline__ void in_sample(const BwdParams& p)
    {
        if (p.kv_lengths) {
            const int given = __builtin_amdgcn_readfirstlane(p.kv_lengths[bh / (uint32_t)p.kv_heads]);
            len = given < 0 ? 0 : given < len ? given : len;
        }
    }
};

// ---------------------------------------------------------------- dk and dv

// What bounds it: the matrix cores together with what feeds them, at the clock
// that the power leaves (1.7 to 1.9 of 2.4 GHz).  They are busy 58 to 60% of the
// cycles, the LDS reads, one fragment a product, and the vector ALU a third each.
// The four products run at 1141 TFLOP/s on 32760 tokens of 5 heads of 128 and at
// 1094 on 4608 of 48, launched alone; a large library product, under the same
// power, reaches 1180 to 1600 by how its operands lie.  Tiles of 64 queries measured 6% faster than
// tiles of 32, and keeping the phases of a block apart 3% more: left to itself
// the scheduler mixes two blocks and has to spill.
//
// head_dim 256 takes all 512 registers of a lane: 256 accumulators, 128 of k and
// v, 32 scores.  The barriers to the scheduler that only it has keep a phase's
// operands from being read in the one before, which would spill.
//
// DS = 2, for head_dim 256: two waves share a block of 32 keys, each with the
// scores of all and half the columns of dk and dv.  That is 6 products for 4, but
// twice the workgroups, for calls that leave CUs idle (8 heads of 512 tokens: 44
// against 55 us; 16 heads of 4096, which do not: 1409 against 1083).
//
// PACKED: with one term and with two in one kernel, both have to fit into the same
// registers: nothing that follows from the lane is shared, and held, by the two, and
// barriers to the scheduler keep the operands of the last products (k = 0 and 1) apart,
// which is also what one term runs best with (sequences of 4096 to 221, 40 heads of 128:
// 1345 us, 1375 without; 2048, 1021, 700, 355, 13 and 1 causal, 40 heads on 8: 362 and 453).
template <int D, bool F16, bool CAUSAL, bool TWO, int DS, bool PACKED>
__device__ __forceinline__ void key_gradients(const BwdParams& p, const Work& w, const char* lds, float* tops)
{
    constexpr int NW = kWaves;
    constexpr int BK = NW / DS * 32, BQ = kTileRows, DB = D / 32 / DS;
    constexpr int QB = PACKED && TWO ? 1 : BQ / 32;       // a tile's rows past kTwoTermRows are nobody's
    constexpr bool kApart = D == 256 || (PACKED && (D == 64 || !TWO));
    constexpr int kTile = BQ * D * 2;
    int lane = threadIdx.x % 64;
    if constexpr (PACKED && TWO)
        __asm__ volatile("" : "+v"(lane));
    const int n = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    const uint32_t bh = w.bh;
    const int64_t b = PACKED ? 0 : bh / (uint32_t)p.kv_heads;
    const int hk = PACKED ? bh : bh % (uint32_t)p.kv_heads;
    const int split = w.split, kb = w.block, seq = w.seq;
    const int q_tokens = w.q_tokens, kv_tokens = w.kv_tokens, len = w.len;
    const int64_t q_at = w.q_at, kv_at = w.kv_at;
    const int shift = kv_tokens - q_tokens;
    const int k0 = kb * BK + wave / DS * 32;              // the wave's first key
    const int key = k0 + n;                               // this lane's
    const int db0 = DS == 1 ? 0 : wave % DS * DB;         // the wave's first column block
    // the first query that sees one of the workgroup's keys, in whole tiles
    int first = 0;
    if (CAUSAL) {
        const int i = kb * BK - shift;
        first = i > 0 ? i / BQ : 0;
    }
    const int tiles = (q_tokens + BQ - 1) / BQ;
    const int per = tiles > first ? tiles - first : 0;    // tiles of one query head
    const int all = kb * BK < len ? per * p.group : 0;
    const int each = (all + p.row_splits - 1) / p.row_splits;
    const int t0 = split * each;
    const int total = (all < t0 + each ? all : t0 + each) - t0;

    f32x16 dk[DB], dv[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i)
        dk[i] = dv[i] = f32x16{};

    // waves 0 and 1 stage the four groups of q's rows, 2 and 3 those of dout's
    static_assert(NW == 4, "two groups of 16 rows a wave");
    const bool stages_q = wave < 2;
    const int64_t stage_ts = stages_q ? p.q_ts : p.do_ts;
    const int64_t stage_hs = stages_q ? p.q_hs : p.do_hs;
    const uint16_t* stage_base = (stages_q ? p.q + b * p.q_bs : p.dout + b * p.do_bs) + q_at * stage_ts;
    const Stager<D> rows(lane, stage_ts);
    const uint32_t lds0 = lds_address(lds);
    uint32_t fill = lds0;
    TileAt at(lds0, lane);

    // the tiles run through the queries of one head of the group after another;
    // h and next_q: the next one to be staged
    int h = hk * p.group + (per ? t0 / per : 0), next_q = (first + (per ? t0 % per : 0)) * BQ;
    const auto stage = [&](int buf) {
        const int left = q_tokens - next_q;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            rows.load(stage_base + (int64_t)next_q * stage_ts + h * stage_hs, stage_ts, left,
                      fill + (stages_q ? 0 : kTile), (wave & 1) * 2 + i);
        if (wave < 2) {           // lse2 and delta: zero past the last query, as are its rows
            const uint64_t a = reinterpret_cast<uint64_t>(
                p.stats + ((b * p.heads + h) * p.q_tokens + q_at + next_q) * 2);
            const u32x4 rsrc = {scalar((uint32_t)a), scalar((uint32_t)(a >> 32) & 0xffffu),
                                scalar((left < BQ ? left : BQ) * 8), kRawBuffer};
            dma4(rsrc, wave * 256 + lane * 4, lds0 + 4 * kTile + buf * BQ * 8 + wave * 256);
        }
        fill ^= 2 * kTile;
        next_q += BQ;
        if (next_q >= q_tokens) {
            next_q = first * BQ;
            ++h;
        }
    };

    int q0 = next_q;
    if (total > 0)
        stage(0);                 // before k and v: the waits run together
    u32x4 kf[D / 16], vf[D / 16];
    {
        const uint16_t* kr = p.k + b * p.k_bs + (kv_at + key) * p.k_ts + hk * p.k_hs + 8 * g;
        const uint16_t* vr = p.v + b * p.v_bs + (kv_at + key) * p.v_ts + hk * p.v_hs + 8 * g;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            kf[kk] = key < len ? load16<false>(kr + 16 * kk) : u32x4{0, 0, 0, 0};
            vf[kk] = key < len ? load16<false>(vr + 16 * kk) : u32x4{0, 0, 0, 0};
        }
    }
    float down = 1.0f;            // brings dp - delta below 1
    int e = 0;
    if constexpr (F16) {
        const int n = p.group * p.stat_blocks;
        float bound;
        if constexpr (PACKED)
            bound = largest_packed<kStatRows>(p.row_norms, (int64_t)hk * p.group, p.group, p.stat_blocks, p.q_rows, seq,
                                              q_tokens, tops) *
                    largest_packed<value_rows(D)>(p.value_norms, hk, 1, p.value_blocks, p.kv_rows, seq, len, tops + 4);
        else
            bound = largest(p.row_norms + bh * n, n, tops) *
                    largest(p.value_norms + bh * p.value_blocks, p.value_blocks, tops + 4);
        e = __builtin_amdgcn_readfirstlane(bound_exponent(bound)) + 1;
        down = __builtin_amdgcn_ldexpf(1.0f, -e);
    }
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        settle(kf[kk]);
        settle(vf[kk]);
    }
    for (int t = 0; t < total; ++t) {
        const int buf = t & 1;
        wait_staged();
        __syncthreads();
        const int following = next_q;
        if (t + 1 < total)
            stage(buf ^ 1);
        const uint32_t st = lds0 + 4 * kTile + buf * BQ * 8 + 32 * g;

#pragma unroll
        for (int y = 0; y < QB; ++y) {
            __builtin_amdgcn_sched_barrier(0);      // one block after the other
            f32x16 s{}, dp{};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                s = mfma<F16>(row_fragment(at, y * block_bytes<D>(), kk), kf[kk], s);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                dp = mfma<F16>(row_fragment(at, kTile + y * block_bytes<D>(), kk), vf[kk], dp);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
                const f32x4 a = *reinterpret_cast<LdsFloats>(st + 256 * y + 64 * i4);
                const f32x4 c = *reinterpret_cast<LdsFloats>(st + 256 * y + 64 * i4 + 16);
                const float lse2[4] = {a[0], a[2], c[0], c[2]};
                const float delta[4] = {a[1], a[3], c[1], c[3]};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 4 * i4 + i;
                    const float pr = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], p.c, -lse2[i]));
                    s[j] = pr;
                    dp[j] = F16 ? pr * ((dp[j] - delta[i]) * down) : pr * (dp[j] - delta[i]);
                }
            }
            if (CAUSAL && __builtin_expect(k0 + 31 > q0 + 32 * y + shift, 0)) {
                keep_branch();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key > q0 + 32 * y + 8 * (i / 4) + 4 * g + i % 4 + shift)
                        s[i] = dp[i] = 0.0f;
            }
            if constexpr (D == 256)
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if constexpr (kApart)
                    __builtin_amdgcn_sched_barrier(0);
                const u32x4 pf = pack_b<F16>(s, k), sf = pack_b<F16>(dp, k);
                u32x4 p_rest, s_rest;
                if constexpr (TWO) {
                    p_rest = pack_rest<F16>(s, k, pf);
                    s_rest = pack_rest<F16>(dp, k, sf);
                }
#pragma unroll
                for (int i = 0; i < DB; ++i) {
                    const u32x4 f = tr_fragment(at, kTile + y * block_bytes<D>() + db0 * kSlab, k, i);
                    dv[i] = mfma<F16>(f, pf, dv[i]);
                    if constexpr (TWO)
                        dv[i] = mfma<F16>(f, p_rest, dv[i]);
                }
#pragma unroll
                for (int i = 0; i < DB; ++i) {
                    const u32x4 f = tr_fragment(at, y * block_bytes<D>() + db0 * kSlab, k, i);
                    dk[i] = mfma<F16>(f, sf, dk[i]);
                    if constexpr (TWO)
                        dk[i] = mfma<F16>(f, s_rest, dk[i]);
                }
            }
        }
        q0 = following;
        at.flip(2 * kTile);
    }

    // the lane's place again: kept over the loop it would take registers that
    // packed sequences and head_dim 256 do not have (nor it, below, for more than one
    // block at a time)
    int lane_now = lane;
    if constexpr (D == 256 || PACKED) {
        lane_now = threadIdx.x % 64;
        __asm__ volatile("" : "+v"(lane_now));
    }
    const int gs = lane_now >> 5, ks = k0 + (lane_now & 31);
    const bool valid = ks < kv_tokens;
    const int64_t to = kv_at + (valid ? ks : kv_tokens - 1);
    const float fv = F16 ? 0x1p-15f : 1.0f;
    const float fk = F16 ? __builtin_amdgcn_ldexpf(p.scale, e - 15) : p.scale;
    const bool seen = ks < len;   // the scores of a padding key are no scores
    if (p.row_splits == 1) {
        uint16_t* kr = p.dk + b * p.dk_bs + to * p.dk_ts + hk * p.dk_hs + 32 * db0;
        uint16_t* vr = p.dv + b * p.dv_bs + to * p.dv_ts + hk * p.dv_hs + 32 * db0;
#pragma unroll
        for (int i = 0; i < DB; ++i) {
            if constexpr (D == 256)
                __builtin_amdgcn_sched_barrier(0);
            store_column<F16>(kr + 32 * i, dk[i], fk, gs, valid, seen);
            store_column<F16>(vr + 32 * i, dv[i], fv, gs, valid, seen);
        }
    } else {
        float* row = p.part_kv + ((split * (int64_t)p.pairs + bh) * p.kv_tokens + to) * 2 * D + 32 * db0;
#pragma unroll
        for (int i = 0; i < DB; ++i) {
            if constexpr (D == 256)
                __builtin_amdgcn_sched_barrier(0);
            store_column_f32(row + 32 * i, dk[i], fk, gs, valid, seen);
            store_column_f32(row + D + 32 * i, dv[i], fv, gs, valid, seen);
        }
    }
}

// ---------------------------------------------------------------- dq

template <int D, bool F16, bool CAUSAL, bool TWO, bool PACKED>
__device__ __forceinline__ void query_gradients(const BwdParams& p, const Work& w, const char* lds, float* tops)
{
    constexpr int NW = kWaves, BN = kTileRows;
    constexpr int BM = NW * 32, KB = BN / 32, DB = D / 32;
    constexpr int kTile = BN * D * 2;
    int lane = threadIdx.x % 64;
    if constexpr (PACKED)         // as in key_gradients
        __asm__ volatile("" : "+v"(lane));
    const int n = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    const uint32_t bh = w.bh;
    const int64_t b = PACKED ? 0 : bh / (uint32_t)p.kv_heads;
    const int hk = PACKED ? bh : bh % (uint32_t)p.kv_heads;
    const int split = w.split, mb = w.block, seq = w.seq;
    const int q_tokens = w.q_tokens, kv_tokens = w.kv_tokens, rows = w.rows, len = w.len;
    const int64_t q_at = w.q_at, kv_at = w.kv_at;
    const int r0 = mb * BM + wave * 32;
    const int r = r0 + n < rows ? r0 + n : rows - 1;
    const int qi = r / p.group, head = hk * p.group + r % p.group;
    const int shift = kv_tokens - q_tokens;
    int end = len;
    if (CAUSAL) {
        const int last = (mb * BM + BM < rows ? mb * BM + BM : rows) - 1;
        const int sees = last / p.group + shift + 1;
        end = sees < end ? (sees < 0 ? 0 : sees) : end;
    }
    const int all = (end + BN - 1) / BN;
    const int each = (all + p.key_splits - 1) / p.key_splits;
    const int t0 = split * each;
    const int tiles = all < t0 + each ? all : t0 + each;
    int open = len;
    if (CAUSAL) {
        const int s = (r0 < rows ? r0 : rows - 1) / p.group + shift + 1;
        open = s < open ? s : open;
    }

    f32x16 dq[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i)
        dq[i] = f32x16{};

    const Stager<D> ks(lane, p.k_ts), vs(lane, p.v_ts);
    const uint16_t* kbase = p.k + b * p.k_bs + kv_at * p.k_ts + hk * p.k_hs;
    const uint16_t* vbase = p.v + b * p.v_bs + kv_at * p.v_ts + hk * p.v_hs;
    uint32_t fill = lds_address(lds);
    TileAt at(fill, lane);
    const auto stage = [&](int t) {
        const int64_t first = (int64_t)t * BN;
#pragma unroll
        for (int i = 0; i < BN / 16 / NW; ++i) {
            ks.load(kbase + first * p.k_ts, p.k_ts, len - (int)first, fill, wave + i * NW);
            vs.load(vbase + first * p.v_ts, p.v_ts, len - (int)first, fill + kTile, wave + i * NW);
        }
        fill ^= 2 * kTile;
    };
    if (t0 < tiles)
        stage(t0);                // before q and dout: the waits run together
    u32x4 qf[D / 16], df[D / 16];
    {
        const uint16_t* qr = p.q + b * p.q_bs + (q_at + qi) * p.q_ts + head * p.q_hs + 8 * g;
        const uint16_t* dr = p.dout + b * p.do_bs + (q_at + qi) * p.do_ts + head * p.do_hs + 8 * g;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            qf[kk] = load16<false>(qr + 16 * kk);
            df[kk] = load16<false>(dr + 16 * kk);
        }
    }
    const f32x2 st = reinterpret_cast<const f32x2*>(p.stats)[(b * p.heads + head) * p.q_tokens + q_at + qi];
    const float delta = st.y;
    int e = 0;
    if constexpr (F16) {
        float sq = 0.0f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            float x[8];
            unpack8<true>(df[kk], x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sq = __builtin_fmaf(x[i], x[i], sq);
        }
        float top;
        if constexpr (PACKED)
            top = largest_packed<value_rows(D)>(p.value_norms, hk, 1, p.value_blocks, p.kv_rows, seq, len, tops);
        else
            top = largest(p.value_norms + bh * p.value_blocks, p.value_blocks, tops);
        e = bound_exponent(sqrtf(half_sum(sq)) * top) + 1;
    }
    // ds alone is needed here, so its power of two goes into the exponent of p
    const float lse2 = st.x + (float)e;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        settle(qf[kk]);
        settle(df[kk]);
    }
    for (int t = t0; t < tiles; ++t) {
        wait_staged();
        __syncthreads();
        if (t + 1 < tiles)
            stage(t + 1);
        const int sees = CAUSAL ? (qi + shift + 1 < len ? qi + shift + 1 : len) : len;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            f32x16 s{}, dp{};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                s = mfma<F16>(row_fragment(at, j * block_bytes<D>(), kk), qf[kk], s);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                dp = mfma<F16>(row_fragment(at, kTile + j * block_bytes<D>(), kk), df[kk], dp);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float pr = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.c, -lse2));
                s[i] = pr * (dp[i] - delta);
            }
            if (__builtin_expect(t * BN + BN > open, 0)) {      // hidden keys: their scores are no scores
                keep_branch();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (t * BN + j * 32 + 8 * (i / 4) + 4 * g + i % 4 >= sees)
                        s[i] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const u32x4 sf = pack_b<F16>(s, k);
                u32x4 s_rest;
                if constexpr (TWO)
                    s_rest = pack_rest<F16>(s, k, sf);
#pragma unroll
                for (int i = 0; i < DB; ++i) {
                    const u32x4 f = tr_fragment(at, j * block_bytes<D>(), k, i);
                    dq[i] = mfma<F16>(f, sf, dq[i]);
                    if constexpr (TWO)
                        dq[i] = mfma<F16>(f, s_rest, dq[i]);
                }
            }
        }
        at.flip(2 * kTile);
    }

    const bool valid = r0 + n < rows;
    const float f = F16 ? __builtin_amdgcn_ldexpf(p.scale, e - 15) : p.scale;
    if (p.key_splits == 1) {
        uint16_t* row = p.dq + b * p.dq_bs + (q_at + qi) * p.dq_ts + head * p.dq_hs;
#pragma unroll
        for (int i = 0; i < DB; ++i)
            store_column<F16>(row + 32 * i, dq[i], f, g, valid);
    } else {
        float* row = p.part_q + ((split * (int64_t)p.pairs + bh) * p.rows + q_at * p.group + r) * D;
#pragma unroll
        for (int i = 0; i < DB; ++i)
            store_column_f32(row + 32 * i, dq[i], f, g, valid);
    }
}

// Both in one launch, dk and dv first (their workgroups take longer): they do
// not wait for each other, so the last workgroups of the one leave no CU idle
// that the other could use.
//
// TWO: p and ds go into the products as two 16-bit terms, the second being what
// the rounding of the first left, so that the gradients are off by their own
// rounding alone.  It is for calls of up to kTwoTermRows rows a key head, which wait
// for memory and launches (16 queries over 32760 keys, 5 heads of 128: 76 us,
// 70 with one term; 2 x 1 over 256, 24 heads of 64: 18 us with either).
constexpr int backward_waves(int d, bool f16, bool two)
{
    // fp16's scaling and both terms together need more than 256 registers
    return d == 256 || (d == 128 && f16 && two) ? 1 : 2;
}

// A workgroup's key block.  Causal: the first key blocks are seen by most queries;
// turning the order from split to split keeps them from meeting on the same CUs.
template <bool CAUSAL>
__device__ __forceinline__ Work key_work(const BwdParams& p, uint32_t bid)
{
    const BlockOf<> block(bid, p.pairs, p.key_blocks * p.row_splits);
    const int split = block.part / p.key_blocks;
    return Work(p, block.pair, split, (block.part + (CAUSAL ? split : 0)) % p.key_blocks);
}

// A workgroup's row block: causal, the longest first.
template <bool CAUSAL>
__device__ __forceinline__ Work query_work(const BwdParams& p, uint32_t bid, bool packed)
{
    const BlockOf<> block(bid, p.pairs, p.row_blocks * p.key_splits);
    const int mb = block.part % p.row_blocks;
    return Work(p, block.pair, block.part / p.row_blocks, CAUSAL && !packed ? p.row_blocks - 1 - mb : mb);
}

template <int D, bool F16, bool CAUSAL, bool TWO>
__global__ __launch_bounds__(kWaves * 64, backward_waves(D, F16, TWO))
void attention_backward_kernel(const BwdParams p)
{
    // two buffers of two tiles, then two of the tiles' lse2 and delta
    constexpr int kTiles = 4 * kTileRows * D * 2;
    __shared__ __attribute__((aligned(kTiles))) char lds[kTiles + 2 * kTileRows * 8];
    __shared__ float tops[8];
    const uint32_t first = p.pairs * (uint32_t)(p.key_blocks * p.row_splits);
    if (blockIdx.x < first) {
        Work w = key_work<CAUSAL>(p, blockIdx.x);
        w.in_sample(p);
        if (D == 256 && p.column_waves == 2)
            key_gradients<D, F16, CAUSAL, TWO, D == 256 ? 2 : 1, false>(p, w, lds, tops);
        else
            key_gradients<D, F16, CAUSAL, TWO, 1, false>(p, w, lds, tops);
    } else {
        Work w = query_work<CAUSAL>(p, blockIdx.x - first, false);
        w.in_sample(p);
        query_gradients<D, F16, CAUSAL, TWO, false>(p, w, lds, tops);
    }
}

// The same of packed sequences, with whole blocks of keys.  Each sequence's own rows
// say how many terms p and ds have, whatever the others are, so both forms are in the
// kernel.
template <int D, bool F16, bool CAUSAL>
__global__ __launch_bounds__(kWaves * 64, backward_waves(D, F16, false))
void packed_backward_kernel(const BwdParams p)
{
    constexpr int kTiles = 4 * kTileRows * D * 2;
    __shared__ __attribute__((aligned(kTiles))) char lds[kTiles + 2 * kTileRows * 8];
    __shared__ float tops[8];
    const uint32_t first = p.pairs * (uint32_t)(p.key_blocks * p.row_splits);
    if (blockIdx.x < first) {
        Work w = key_work<CAUSAL>(p, blockIdx.x);
        const PackedBlock<kWaves * 32> of(p, p.kv_rows, 1, w.block);
        if (!of.there(p, of.kv_tokens))
            return;
        w.in_sequence(p, of);
        if (p.q_rows.rest(w.seq))
            w.q_tokens = w.rows = 0;
        if (w.q_tokens == 0)
            w.len = 0;
        if (w.rows <= kTwoTermRows)
            key_gradients<D, F16, CAUSAL, true, 1, true>(p, w, lds, tops);
        else
            key_gradients<D, F16, CAUSAL, false, 1, true>(p, w, lds, tops);
    } else {
        Work w = query_work<CAUSAL>(p, blockIdx.x - first, true);
        const PackedBlock<kWaves * 32> of(p, p.q_rows, p.group, w.block);
        if (!of.there(p, of.q_tokens * p.group))
            return;
        w.in_sequence(p, of);
        if (p.q_rows.rest(w.seq))
            w.kv_tokens = 0;
        if (CAUSAL)
            w.block = (w.rows + kWaves * 32 - 1) / (kWaves * 32) - 1 - w.block;
        if (w.rows <= kTwoTermRows)
            query_gradients<D, F16, CAUSAL, true, true>(p, w, lds, tops);
        else
            query_gradients<D, F16, CAUSAL, false, true>(p, w, lds, tops);
    }
}

// Rows that have parts to add, and the workgroups that add them.
template <bool KV>
__host__ __device__ __forceinline__ int64_t part_rows(const BwdParams& p)
{
    return (int64_t)p.pairs * (KV ? 2 * (int64_t)p.kv_tokens : p.rows);
}

template <int D, bool KV>
__host__ __device__ __forceinline__ int64_t sum_blocks(const BwdParams& p)
{
    constexpr int R = 256 / (D / 8);
    return (KV ? p.row_splits : p.key_splits) > 1 ? (part_rows<KV>(p) + R - 1) / R : 0;
}

// Adds the splits' dk and dv, or dq, in order: D / 8 threads a row.
template <int D, bool F16, bool KV, bool PACKED>
__device__ __forceinline__ void sum_parts(const BwdParams& p, int64_t block)
{
    constexpr int L = D / 8, R = 256 / L;
    const int64_t rows = part_rows<KV>(p);
    const int64_t at = block * R + threadIdx.x / L;
    if (at >= rows)
        return;
    if constexpr (PACKED) {                // rows of no sequence may have to be left alone
        const Rows& of = KV ? p.kv_rows : p.q_rows;
        const int64_t token = KV ? at / 2 % p.kv_tokens : at % p.rows / p.group;
        if (!p.fill_rest && (token < of.first(1) || token >= of.first(of.sequences + 1)))
            return;
    }
    const int d0 = threadIdx.x % L * 8;
    const float* part = (KV ? p.part_kv : p.part_q) + at * D + d0;
    const int splits = KV ? p.row_splits : p.key_splits;
    float s[8] = {};
#pragma unroll 4
    for (int i = 0; i < splits; ++i) {
        float f[8];
        load_f32x8(part + i * rows * D, f);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] += f[j];
    }
    uint16_t* to;
    if constexpr (KV) {
        const int64_t key = at / 2 % p.kv_tokens, bh = at / 2 / p.kv_tokens;
        const int64_t b = bh / p.kv_heads, h = bh % p.kv_heads;
        to = at % 2 ? p.dv + b * p.dv_bs + key * p.dv_ts + h * p.dv_hs
                    : p.dk + b * p.dk_bs + key * p.dk_ts + h * p.dk_hs;
    } else {
        const int64_t bh = at / p.rows, b = bh / p.kv_heads;
        const int r = at % p.rows;
        to = p.dq + b * p.dq_bs + r / p.group * p.dq_ts + (bh % p.kv_heads * p.group + r % p.group) * p.dq_hs;
    }
    store16<false>(to + d0, pack8<F16>(s));
}

// Both in one launch, as calls that have both are small ones, where a launch counts
// (packed 1021, 64, 333, 1, 517 and 128 tokens, 12 heads on 4 of 64, causal: 42.6 us, with
// two launches 45.9; 2 x 1024 tokens, 8 heads of 128: 57.7 and 59.8).
template <int D, bool F16, bool PACKED>
__global__ __launch_bounds__(256)
void attention_sum_kernel(const BwdParams p)
{
    const int64_t first = sum_blocks<D, true>(p);
    if ((int64_t)blockIdx.x < first)
        sum_parts<D, F16, true, PACKED>(p, blockIdx.x);
    else
        sum_parts<D, F16, false, PACKED>(p, blockIdx.x - first);
}

// ---------------------------------------------------------------- launches

// How a call is cut up, and where its workspace's parts begin (in floats).
struct Shape {
    int64_t row_blocks, key_blocks, column_waves, row_splits, key_splits;
    int64_t stat_blocks, value_blocks;
    int64_t row_norms, value_norms, part_kv, part_q, floats;
};

// The splits of at most `tiles` tiles that let `blocks` workgroups fill a chip
// that holds `resident`: none if they fill half of it, and runs of at least
// `least` tiles (about 10 us of work, twice what the launch that adds them
// costs).  A workgroup divides the tiles that its masks leave.
int64_t splits_of(int64_t blocks, int64_t resident, int64_t tiles, int64_t least)
{
    if (blocks == 0 || 2 * blocks > resident || tiles < 2 * least)
        return 1;
    const int64_t fill = resident / blocks, most = tiles / least;
    return fill < most ? fill : most;
}

// Packed sequences (`packed`; a's sizes are the buffers') are cut as one sequence of
// all rows would be: a workgroup divides what its own sequence leaves.
Shape shape_of(const dit_attn_args& a, const dit_attn_packed_args* packed)
{
    Shape s;
    const int64_t group = a.heads / a.kv_heads, rows = a.q_tokens * group;
    const int64_t pairs = a.batch * a.kv_heads;
    constexpr int64_t per = 32 * kWaves;
    const auto blocks_of = [&](int64_t n, int64_t size) {
        return packed ? qkr_attn_host::blocks_of(n, packed->sequences, size) : (n + size - 1) / size;
    };
    s.row_blocks = blocks_of(rows, per);
    // workgroups resident at once (head_dim 64 would hold 3 a CU, but its sums of
    // more parts cost what that gains: 33 us with 2 as with 3 on 12 x 8 blocks)
    const int64_t resident = 256 * (a.head_dim == 256 ? 1 : 2);
    s.key_splits = splits_of(pairs * s.row_blocks, resident, (a.kv_tokens + 63) / 64, 8);
    // head_dim 256: two waves to a block of keys if all workgroups still run at once
    for (s.column_waves = a.head_dim == 256 && !packed ? 2 : 1;; s.column_waves = 1) {
        const int64_t keys = per / s.column_waves;
        s.key_blocks = blocks_of(a.kv_tokens, keys);
        s.row_splits = splits_of(pairs * s.key_blocks, resident, (a.q_tokens + 63) / 64 * group, 8);
        if (s.column_waves == 1 ||
            pairs * (s.key_blocks * s.row_splits + s.row_blocks * s.key_splits) <= resident)
            break;
    }
    s.stat_blocks = blocks_of(a.q_tokens, kStatRows);
    s.value_blocks = blocks_of(a.kv_tokens, value_rows(a.head_dim));
    const auto whole = [](int64_t n) { return (n + 3) / 4 * 4; };
    s.row_norms = whole(a.batch * a.heads * a.q_tokens * 2);
    s.value_norms = s.row_norms + whole(a.batch * a.heads * s.stat_blocks);
    s.part_kv = s.value_norms + whole(pairs * s.value_blocks);
    s.part_q = s.part_kv + (s.row_splits > 1 ? s.row_splits * pairs * a.kv_tokens * 2 * a.head_dim : 0);
    s.floats = s.part_q + (s.key_splits > 1 ? s.key_splits * pairs * rows * a.head_dim : 0);
    return s;
}

template <int D, bool F16, bool CAUSAL, bool PACKED>
hipError_t launch(BwdParams p, hipStream_t st)
{
    const int64_t pairs = p.pairs;
    void* argv[] = {&p};
    hipError_t err = hipSuccess;
    const auto go = [&](auto fn, int64_t blocks) {
        if (err == hipSuccess && blocks)
            err = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)blocks), dim3(256),
                                  argv, 0, st);
    };
    go(row_stats_kernel<D, F16, PACKED>, p.batch * p.heads * p.stat_blocks + (F16 ? pairs * p.value_blocks : 0));
    go(PACKED                   ? packed_backward_kernel<D, F16, CAUSAL>
       : p.rows <= kTwoTermRows ? attention_backward_kernel<D, F16, CAUSAL, true>
                                : attention_backward_kernel<D, F16, CAUSAL, false>,
       pairs * ((int64_t)p.key_blocks * p.row_splits + (int64_t)p.row_blocks * p.key_splits));
    go(attention_sum_kernel<D, F16, PACKED>, sum_blocks<D, true>(p) + sum_blocks<D, false>(p));
    return err;
}

template <int D, bool PACKED>
hipError_t launch(const BwdParams& p, bool f16, bool causal, hipStream_t st)
{
    if (f16)
        return causal ? launch<D, true, true, PACKED>(p, st) : launch<D, true, false, PACKED>(p, st);
    return causal ? launch<D, false, true, PACKED>(p, st) : launch<D, false, false, PACKED>(p, st);
}

template <int D>
hipError_t launch(const BwdParams& p, bool f16, bool causal, bool packed, hipStream_t st)
{
    return packed ? launch<D, true>(p, f16, causal, st) : launch<D, false>(p, f16, causal, st);
}

// Both entry points, after the checks of their sizes.
int backward(const dit_attn_args& a, const dit_attn_packed_args* packed, const dit_attn_tensor* dout,
             const dit_attn_tensor* q, const dit_attn_tensor* k, const dit_attn_tensor* v,
             const dit_attn_tensor* out, const float* lse, const dit_attn_tensor* dq, const dit_attn_tensor* dk,
             const dit_attn_tensor* dv, void* workspace, int64_t workspace_bytes, void* stream)
{
    using namespace qkr_attn_host;
    int rc;
    const Extent eq = {a.q_tokens, a.heads}, ekv = {a.kv_tokens, a.kv_heads};
    const struct { dit_attn_tensor t; Extent e; } all[] = {
        {plain(a, dout, eq), eq}, {plain(a, q, eq), eq}, {plain(a, k, ekv), ekv}, {plain(a, v, ekv), ekv},
        {plain(a, out, eq), eq}, {plain(a, dq, eq), eq}, {plain(a, dk, ekv), ekv}, {plain(a, dv, ekv), ekv}};
    for (int i = 0; i < 8; ++i)
        if ((rc = check_tensor(a, all[i].t, all[i].e, i >= 5)))
            return rc;
    if (a.q_tokens && !lse)
        return QKR_ERR_NULL;
    const Lengths lengths(a, packed);
    if (reinterpret_cast<uintptr_t>(lse) & 3u || !lengths.aligned())
        return QKR_ERR_ALIGN;
    const int64_t need = shape_of(a, packed).floats * 4;
    if (need && (!workspace || workspace_bytes < need))
        return QKR_ERR_WORKSPACE;
    if (!qkr_host::aligned16(workspace))
        return QKR_ERR_ALIGN;
    const Range lse_r = {lse, (uint64_t)a.batch * a.heads * a.q_tokens * 4};
    const Range ws_r = {workspace, (uint64_t)need};
    if (meet(ws_r, lse_r) || meet(ws_r, lengths.range[0]) || meet(ws_r, lengths.range[1]))
        return QKR_ERR_ARG;
    for (int i = 0; i < 8; ++i) {
        const Range x = range(a, all[i].t, all[i].e);
        if (meet(x, ws_r))
            return QKR_ERR_ARG;
        if (i < 5)
            continue;
        if (meet(x, lse_r) || meet(x, lengths.range[0]) || meet(x, lengths.range[1]))
            return QKR_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (may_meet(a, all[i].t, all[i].e, all[j].t, all[j].e))
                return QKR_ERR_ARG;
    }

    BwdParams p = {};
    unpack(all[0].t, p.dout, p.do_bs, p.do_ts, p.do_hs);
    unpack(all[1].t, p.q, p.q_bs, p.q_ts, p.q_hs);
    unpack(all[2].t, p.k, p.k_bs, p.k_ts, p.k_hs);
    unpack(all[3].t, p.v, p.v_bs, p.v_ts, p.v_hs);
    unpack(all[4].t, p.out, p.o_bs, p.o_ts, p.o_hs);
    unpack(all[5].t, p.dq, p.dq_bs, p.dq_ts, p.dq_hs);
    unpack(all[6].t, p.dk, p.dk_bs, p.dk_ts, p.dk_hs);
    unpack(all[7].t, p.dv, p.dv_bs, p.dv_ts, p.dv_hs);
    p.lse = lse;
    p.kv_lengths = a.kv_lengths;
    if (packed) {
        p.q_rows = Rows{packed->q_offsets, (int32_t)packed->sequences, (int32_t)a.q_tokens};
        p.kv_rows = Rows{packed->kv_offsets ? packed->kv_offsets : packed->q_offsets, (int32_t)packed->sequences,
                         (int32_t)a.kv_tokens};
        p.fill_rest = packed->fill_rest;
    }
    p.batch = a.batch;
    p.pairs = (uint32_t)(a.batch * a.kv_heads);
    p.q_tokens = (int32_t)a.q_tokens;
    p.kv_tokens = (int32_t)a.kv_tokens;
    p.heads = a.heads;
    p.kv_heads = a.kv_heads;
    p.group = a.heads / a.kv_heads;
    p.rows = (int32_t)(a.q_tokens * p.group);
    p.scale = a.scale;
    p.c = a.scale * kLog2e;
    p.stats = static_cast<float*>(workspace);
    const Shape shape = shape_of(a, packed);
    p.row_blocks = (int32_t)shape.row_blocks;
    p.key_blocks = (int32_t)shape.key_blocks;
    p.column_waves = (int32_t)shape.column_waves;
    p.row_splits = (int32_t)shape.row_splits;
    p.key_splits = (int32_t)shape.key_splits;
    p.stat_blocks = (int32_t)shape.stat_blocks;
    p.value_blocks = (int32_t)shape.value_blocks;
    p.row_norms = p.stats + shape.row_norms;
    p.value_norms = p.stats + shape.value_norms;
    p.part_kv = p.stats + shape.part_kv;
    p.part_q = p.stats + shape.part_q;
    const bool f16 = a.dtype == QKR_FP16, causal = a.causal != 0;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t err = a.head_dim == 64    ? launch<64>(p, f16, causal, packed, st)
                           : a.head_dim == 128 ? launch<128>(p, f16, causal, packed, st)
                                               : launch<256>(p, f16, causal, packed, st);
    return err == hipSuccess ? QKR_OK : QKR_ERR_HIP;
}

}  // namespace

extern "C" int64_t dit_attention_backward_workspace_size(const dit_attn_args* args)
{
    const int rc = qkr_attn_host::check_args(args);
    return rc != QKR_OK ? rc : shape_of(*args, nullptr).floats * 4;
}

extern "C" int dit_attention_backward(const dit_attn_args* args, const dit_attn_tensor* dout,
                                      const dit_attn_tensor* q, const dit_attn_tensor* k,
                                      const dit_attn_tensor* v, const dit_attn_tensor* out,
                                      const float* lse, const dit_attn_tensor* dq,
                                      const dit_attn_tensor* dk, const dit_attn_tensor* dv,
                                      void* workspace, int64_t workspace_bytes, void* stream)
{
    const int rc = qkr_attn_host::check_args(args);
    if (rc != QKR_OK || args->batch == 0 || (args->q_tokens == 0 && args->kv_tokens == 0))
        return rc;
    return backward(*args, nullptr, dout, q, k, v, out, lse, dq, dk, dv, workspace, workspace_bytes, stream);
}

extern "C" int64_t dit_attention_packed_backward_workspace_size(const dit_attn_packed_args* args)
{
    dit_attn_args a;
    const int rc = qkr_attn_host::check_packed(args, a);
    return rc != QKR_OK ? rc : shape_of(a, args).floats * 4;
}

extern "C" int dit_attention_packed_backward(const dit_attn_packed_args* args, const dit_attn_tensor* dout,
                                             const dit_attn_tensor* q, const dit_attn_tensor* k,
                                             const dit_attn_tensor* v, const dit_attn_tensor* out,
                                             const float* lse, const dit_attn_tensor* dq,
                                             const dit_attn_tensor* dk, const dit_attn_tensor* dv,
                                             void* workspace, int64_t workspace_bytes, void* stream)
{
    dit_attn_args a;
    const int rc = qkr_attn_host::check_packed(args, a);
    if (rc != QKR_OK || (a.q_tokens == 0 && a.kv_tokens == 0))
        return rc;
    if (!args->q_offsets)
        return QKR_ERR_NULL;
    return backward(a, args, dout, q, k, v, out, lse, dq, dk, dv, workspace, workspace_bytes, stream);
}
