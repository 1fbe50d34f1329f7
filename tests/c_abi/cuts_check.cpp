// How the feed-forward products of a call are cut: compiled by
// tests/test_feed_forward_cuts_cpu.py and run on the CPU.  Reads lines of rows,
// hidden, inner and bytes a number; prints for each product (forward, dx, dw) the
// side of its tiles, their number and the splits of k, then the terms of dgate and dup.
#include <stdio.h>

#include "feed_forward_host.h"

static void show(const qkr_ff_host::Cut& c)
{
    printf("%d %lld %lld ", c.large ? 256 : 128, (long long)(c.row_tiles * c.column_tiles), (long long)c.splits);
}

int main()
{
    long long rows, hidden, inner, size;
    while (scanf("%lld %lld %lld %lld", &rows, &hidden, &inner, &size) == 4) {
        show(qkr_ff_host::cut_of(rows, 2 * inner, (hidden * size + 127) / 128, false));
        const dit_ff_args a = {rows, (int32_t)hidden, (int32_t)inner, DIT_FF_SILU, QKR_BF16, QKR_BF16};
        const int terms = qkr_ff_host::terms_of(a);
        show(qkr_ff_host::cut_of(terms * rows, hidden, 2 * ((inner + 63) / 64), true));
        show(qkr_ff_host::cut_of(2 * inner, hidden, (terms * rows + 63) / 64, true));
        printf("%d\n", terms);
    }
    return 0;
}
