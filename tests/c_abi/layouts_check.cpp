// What attention's argument checks say of two tensors' memory, against a count
// of every element: compiled with g++ by tests/test_attention_layouts_cpu.py and
// run on the CPU.  Prints "ok" and exits 0 when no answer is wrong.
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <random>
#include <set>
#include <vector>

#include "attention_host.h"

using qkr_attn_host::Extent;

namespace {

constexpr int kDim = 64;
char* const kAt = reinterpret_cast<char*>(uintptr_t{1} << 40);

// The runs of 8 elements that a tensor holds.
std::set<int64_t> runs(const dit_attn_args& a, const dit_attn_tensor& t, const Extent& e)
{
    std::set<int64_t> all;
    const int64_t at = (static_cast<char*>(t.data) - kAt) / 2;
    for (int64_t b = 0; b < a.batch; ++b)
        for (int64_t i = 0; i < e.tokens; ++i)
            for (int64_t h = 0; h < e.heads; ++h)
                for (int64_t d = 0; d < kDim; d += 8)
                    all.insert((at + b * t.batch_stride + i * t.token_stride + h * t.head_stride + d) / 8);
    return all;
}

bool share(const std::set<int64_t>& x, const std::set<int64_t>& y)
{
    return std::any_of(x.begin(), x.end(), [&](int64_t r) { return y.count(r) > 0; });
}

bool said(const dit_attn_args& a, const dit_attn_tensor& x, const Extent& ex, const dit_attn_tensor& y,
          const Extent& ey)
{
    return qkr_attn_host::may_meet(a, qkr_attn_host::plain(a, &x, ex), ex, qkr_attn_host::plain(a, &y, ey), ey);
}

int wrong(const char* what, const dit_attn_args& a, const dit_attn_tensor& x, const Extent& ex,
          const dit_attn_tensor& y, const Extent& ey)
{
    printf("%s: batch %lld", what, (long long)a.batch);
    for (const auto& [t, e] : {std::pair{x, ex}, std::pair{y, ey}})
        printf("; %lld tokens, %d heads at %lld, strides %lld %lld %lld", (long long)e.tokens, e.heads,
               (long long)(static_cast<char*>(t.data) - kAt) / 2, (long long)t.batch_stride,
               (long long)t.token_stride, (long long)t.head_stride);
    printf("\n");
    return 1;
}

}  // namespace

int main()
{
    std::mt19937 rng(1);
    const auto below = [&](int64_t n) { return (int64_t)(rng() % (uint64_t)n); };
    int apart = 0, joined = 0, told = 0;

    // slices of a buffer whose dimensions (batch, token, slot of a head, tensor,
    // element) stand in any order, heads of either tensor and their places at
    // random: the answer is exact
    for (int n = 0; n < 20000; ++n) {
        dit_attn_args a = {};
        a.batch = 1 + below(3);
        a.head_dim = kDim;
        const int64_t tokens = 1 + below(5), slots = 1 + below(4), tensors = 1 + below(4);
        int64_t size[4] = {a.batch, tokens, slots, tensors}, stride[4], order[4] = {0, 1, 2, 3};
        int64_t s = kDim + 8 * below(2);
        std::shuffle(order, order + 4, rng);
        for (int i : order) {
            stride[i] = s;
            s *= size[i];
        }
        dit_attn_tensor t[2];
        Extent e[2];
        for (int i = 0; i < 2; ++i) {
            const int64_t first = below(slots), token = below(tokens);
            e[i] = Extent{1 + below(tokens - token), (int32_t)(1 + below(slots - first))};
            // now and then a few elements off its place
            const int64_t at = below(tensors) * stride[3] + first * stride[2] + token * stride[1] +
                               (below(4) ? 0 : 8 * below(9));
            t[i] = dit_attn_tensor{kAt + 2 * at, stride[0], stride[1], stride[2]};
        }
        const bool meet = share(runs(a, t[0], e[0]), runs(a, t[1], e[1]));
        if (said(a, t[0], e[0], t[1], e[1]) != meet || said(a, t[1], e[1], t[0], e[0]) != meet)
            return wrong(meet ? "shared" : "apart", a, t[0], e[0], t[1], e[1]);
        ++(meet ? joined : apart);
    }

    // rows beside rows: of one token each, one of them the same for all samples
    for (int64_t tokens : {1, 4})
        for (int64_t single : {0, 1}) {
            dit_attn_args a = {};
            a.batch = 3;
            a.head_dim = kDim;
            const Extent ex = {single ? 1 : tokens, 2}, ey = {tokens, 3};
            const int64_t row = 5 * kDim;
            const dit_attn_tensor x = {kAt + 2 * row, 0, row, kDim};
            const dit_attn_tensor y = {kAt + 2 * (2 * kDim), tokens * row, row, kDim};
            if (said(a, x, ex, y, ey) || said(a, y, ey, x, ex))
                return wrong("apart", a, x, ex, y, ey);
        }

    // any strides (odd and negative ones of single elements too), zeros and ones
    // that fold onto themselves among them: never
    // apart where they share
    for (int n = 0; n < 40000; ++n) {
        dit_attn_args a = {};
        a.batch = 1 + below(3);
        a.head_dim = kDim;
        dit_attn_tensor t[2];
        Extent e[2];
        const bool alike = below(2);
        for (int i = 0; i < 2; ++i) {
            e[i] = Extent{1 + below(4), (int32_t)(1 + below(4))};
            t[i] = dit_attn_tensor{kAt + 16 * below(200), 8 * below(80), kDim + 8 * below(60), 8 * below(40)};
            if (i && alike)
                t[1] = dit_attn_tensor{t[1].data, t[0].batch_stride, t[0].token_stride, t[0].head_stride};
        }
        for (int i = 0; i < 2; ++i) {
            if (a.batch == 1 && below(2))
                t[i].batch_stride = -3;
            if (e[i].tokens == 1 && below(2))
                t[i].token_stride = 5242881;
            if (e[i].heads == 1 && below(2))
                t[i].head_stride = INT64_MIN;
        }
        const bool meet = share(runs(a, t[0], e[0]), runs(a, t[1], e[1]));
        if (meet && (!said(a, t[0], e[0], t[1], e[1]) || !said(a, t[1], e[1], t[0], e[0])))
            return wrong("shared", a, t[0], e[0], t[1], e[1]);
        told += !meet && !said(a, t[0], e[0], t[1], e[1]);
    }
    if (apart < 5000 || joined < 5000 || told < 1000) {
        printf("one-sided: %d apart, %d joined, %d told\n", apart, joined, told);
        return 1;
    }
    printf("ok\n");
    return 0;
}
