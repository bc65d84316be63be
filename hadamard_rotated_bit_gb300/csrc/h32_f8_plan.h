// Which kernel and tile an 8-bit floating-point product runs on: rules on its sizes and the number
// of SMs, host arithmetic alone.
#pragma once

#include <stdint.h>

namespace h32 {

constexpr int64_t kRowsTokens = 32;   // dense: up to here rows_kernel
constexpr int kRowsPerSm = 2;         // rows_kernel: CTAs of an SM at most

// A product's sizes as the kernels number them: rows and tiles in int (a group starts up to 3 rows
// early: at most two chunks more than its rows fill).
inline bool f8_sizes_fit(int64_t M, int64_t N, int64_t K, int64_t E) {
    constexpr int64_t kMost = 0x7FFFFFFFll - 256;
    return M >= 0 && M <= kMost && N > 0 && N <= kMost / E && K > 0 && K <= kMost && K % 32 == 0 &&
           (N + 127) / 128 * (M / 16 + 2 * E) <= 0x7FFFFFFFll;
}

// CTAs that rows_kernel deals a tile's K steps to.  With few tiles a share of at least 4 steps
// each, as long as all of them run at once.  (5120 x 5120 and 7 tokens: one CTA a tile 13.9 us, 4
// 9.4.)
inline int rows_cluster(int64_t tiles, int64_t nb, int sms) {
    int c = 1;
    while (2 * c <= 8 && tiles * 2 * c <= kRowsPerSm * int64_t(sms) && nb >= 8 * c) c *= 2;
    return c;
}

// How lanes_kernel takes `chunks` chunks of tokens (as the host knows them) with so many units
// (CTAs or pairs).  A K step of 64, 128 and 256 weight rows takes a pair 332, 355 and 406 ns (256
// tokens x 5120 x 8192 and 16384; 192 rows 444, so never), a tile's end about 3 us for 256
// rows.  The narrow ones pay where they fill units that were idle (256 tokens x 8192 x 5120: 128
// rows 29.5 us, 256 rows 33.6), and equal runs of K steps where the last wave of whole tiles is
// long (333 x 5120 x 17408: 40 tiles on 76 pairs, 64 and 48 us; 1000 tokens 80); they cost about
// 14 us (clearing the flags, two ends of tiles in turn) and 3.2 for each partial
// sum of a tile.
struct TilePlan {
    int bn;         // weight rows of a tile; 0: rows_kernel
    int runs;       // > 0: runs of K steps for so many pairs, 12 steps at least
    int64_t cost;   // ns, without the launch
};
inline TilePlan plan_tiles(int64_t chunks, int64_t N, int64_t K, int units, bool may_run) {
    const int64_t nb = (K + 127) / 128;
    const auto cost = [&](int64_t bn, int64_t step) {
        const int64_t tiles = (N + bn - 1) / bn * chunks;
        return (tiles + units - 1) / units * (nb * step + 12 * bn);
    };
    const int64_t c64 = cost(64, 332), c128 = cost(128, 355), c256 = cost(256, 406);
    const int64_t best = c256 <= c128 && c256 <= c64 ? c256 : c128 <= c64 ? c128 : c64;
    const int64_t tiles = (N + 255) / 256 * chunks, steps = tiles * nb;
    TilePlan p{best == c256 ? 256 : best == c128 ? 128 : 64, 0, best};
    // (not where every pair has many tiles: the runs then walk all weights at once, which no
    // longer fit the L2; 2048 x 34816 x 5120 read them seven times)
    if (!may_run || steps >= 0x7FFFFFFFll || tiles > 4 * int64_t(units)) return p;
    for (int64_t n = steps / 12 < units ? steps / 12 : units; n >= 2; n = n * 3 / 4) {
        const int64_t run = (steps + n - 1) / n;
        const int64_t c = run * 406 + (tiles / n + 1) * (12 * 256) + 14000 + 3200 * ((nb + run - 1) / run);
        if (c < p.cost) {
            p.cost = c;
            p.runs = static_cast<int>(n);
        }
    }
    return p;
}

// Dense products of more tokens than rows_kernel has columns.  One CTA a tile up to 128 tokens, a
// pair beyond.  Where the tiles are few and K is long, rows_kernel is faster with a tile for
// each 32 tokens, as its clusters share K out: its steps take 430 ns of a CTA and its start 5 us
// more than the other kernel's (128 x 783 x 8896 12.0 us, on the lanes 26.1; 64 x 5120 x 17408 37
// and 47; 512 x 512 x 4096 12.5 and 15.3; but 723 x 418 x 1568 12.4 and 9.2).
inline TilePlan plan_dense(int64_t M, int64_t N, int64_t K, int sms) {
    const bool one = M <= 128;
    TilePlan p = plan_tiles(one ? 1 : (M + 255) / 256, N, K, one ? sms : sms / 2, !one);
    const int64_t nb = (K + 127) / 128;
    const int c = rows_cluster((N + 127) / 128 * ((M + 31) / 32), nb, sms);
    const int64_t rows = 5000 + 430 * ((nb + c - 1) / c);
    return c > 1 && rows < p.cost ? TilePlan{0, 0, rows} : p;
}

struct F8Plan {
    int columns;     // rows_kernel: tokens of a tile, 16 or 32; 0: lanes_kernel
    int cluster;     // rows_kernel: CTAs of a tile
    int bn, ctas;    // lanes_kernel: weight rows of a tile and its CTAs
    int runs;        // lanes_kernel: > 0: runs of K steps for so many pairs, with a workspace
    int64_t tiles;   // whole tiles (of experts: at most)
};

// Tokens of a group, as far as the host knows them, decide the kernel.  Dense, 34816 x
// 5120: 16 tokens as columns 34 us, on the lanes 41; 32 tokens 39 and 35, but 5120 x 17408 25
// and 47 (K shared out over a cluster).  Experts (128 of 1536 x 2048) with 4, 16 and 32
// tokens on average: 16 columns 67, 101 and 151 us, lanes 74, 76 and 77 (groups differ, and a
// second chunk of columns reads the weights again).
// Experts: up to 96 tokens on average one CTA a tile, two beyond, as of 256 rows of a pair the
// half without tokens would idle (64 tokens an expert: 80 and 104 us); dense, 100 x 34816 x 5120:
// 36 and 45, but 4096 x 34816 x 5120 the other way, as a pair reads its weights once.
inline F8Plan plan_f8(int64_t M, int64_t N, int64_t K, int64_t E, bool experts, int sms) {
    const int64_t per = (M + E - 1) / E, nb = (K + 127) / 128, nt = (N + 127) / 128;
    const auto rows = [&](int columns, int64_t tiles) {
        return F8Plan{columns, experts ? 1 : rows_cluster(tiles, nb, sms), 0, 0, 0, tiles};
    };
    if (per <= (experts ? 8 : 16)) return rows(16, nt * E);
    const bool one = per <= (experts ? 96 : 128);
    const int64_t high = one ? 128 : 256, chunks = experts ? E + M / high : (M + high - 1) / high;
    const TilePlan p = experts ? plan_tiles(chunks, N, K, one ? sms : sms / 2, false) : plan_dense(M, N, K, sms);
    if (!experts && (per <= kRowsTokens || p.bn == 0)) return rows(32, nt * ((M + 31) / 32));
    return F8Plan{0, 1, p.bn, one ? 1 : 2, p.runs, (N + p.bn - 1) / p.bn * chunks};
}

}  // namespace h32
