// Which kernel, tiles and stretches an 8-bit matrix product takes, from its sizes alone.  Plain C++, so that a host compiler
// takes it by itself (the tests ask it which kernel their sizes reach).
#pragma once

#include <algorithm>
#include <cstddef>

#include "rs.h"

namespace rs {

constexpr int kBlock = RS_FP8_BLOCK;
constexpr int kSms = 152;
constexpr int kPairs = kSms / 2;

inline int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

struct Plan {
    int rows;      // 16, 32 or 64: few rows, that many columns of products; 0: the tile kernel
    int bn, splits, tiles_n, tiles;
    size_t workspace() const {
        return rows == 0 && splits > 1 ? size_t(splits) * tiles * 2 * bn * 128 * sizeof(float) : 0;
    }
};

// Which kernel and which tiles.
//  - Up to 64 rows the rows kernel (64 x 4096 x 4096: 10.4 us; at 128 rows it took 33.8 us and the tiles 15.2).  The rule
//    looks at that alone: with few columns and a long contraction 64 rows lose to 65 on split tiles (x 256 x 160000
//    107 against 31 us, x 512 x 160000 109 against 43).
//  - 256 columns a tile move the fewest bytes and cost the fewest instructions a product, but with few tiles and
//    little work for each pair of SMs, 128 columns spread it further: 2000 x 1000 x 2000 (32 wide tiles, 7 blocks a
//    pair) 11.7 against 16.5 us, 1000 x 1000 x 3000 14.7 against 17.7; with more of either the other way, 4000 x 1000
//    x 700 (64 tiles) 10.9 against 9.4, 2000 x 700 x 10000 (25 blocks a pair) 41.2 against 33.3.  With one wide tile
//    the split sums count: 256 x 256 x 160000 35 against 38 to 40 us; with two (512 x 256 x 160000) both take 45, and
//    128 columns half of the workspace.
//  - Fewer tiles than pairs: the blocks are split among them, at least 8 to a stretch (256 x 256 x 20000 17 us, with
//    4 19 to 20, with 16 19).
inline Plan plan_matmul(int m, int n, int k) {
    Plan p{};
    const int blocks = ceil_div(k, kBlock);
    if (m <= 64) {
        p.rows = m <= 16 ? 16 : m <= 32 ? 32 : 64;
        p.bn = 128;
        p.tiles_n = p.tiles = ceil_div(n, 128);
        // as many CTAs as two on each SM, of one cluster of eight at most to a tile, with at least two blocks to a CTA:
        // narrow results (up to 2304 columns) leave SMs idle however long the contraction is
        for (p.splits = 1; p.splits < 8 && p.tiles * p.splits * 2 <= 2 * kSms && blocks >= p.splits * 4;) p.splits *= 2;
        return p;
    }
    const long long wide = (long long)ceil_div(m, 256) * ceil_div(n, 256);
    const bool narrow = wide < kPairs / 2 && (wide * blocks <= 10 * kPairs || wide <= 2);
    p.bn = n <= 128 || narrow ? 128 : 256;
    p.tiles_n = ceil_div(n, p.bn);
    const long long tiles = (long long)ceil_div(m, 256) * p.tiles_n;
    p.tiles = int(std::min<long long>(tiles, 0x7fffffff));
    p.splits = tiles >= kPairs ? 1 : std::max(1, std::min(kPairs / p.tiles, blocks / 8));
    return p;
}

// Whether a product with an 8-bit result is the tile kernel's alone: a thread of it holds a row's 128 sums of one block in
// 256 columns a tile, unsplit.  Otherwise the result goes to the workspace in float32 and from there to 8 bits, in two
// more launches at most.
//  - From 65 rows on alone, unless the plan splits a contraction of more than 16 blocks: 160,000 x 512 x 512 58 against
//    180 us, x 128 x 512 31 against 53, 1000 x 512 x 512 6.6 against 8.8 in a graph, 256 x 2048 x 2048 12.3 against 16.6;
//    the other way 512 x 256 x 9300 36 against 17.
//  - Fewer rows alone up to 8 blocks, where a call costs the host 10 us instead of 14 to 16.  On the GPU, in a graph, that
//    is right from about 37 rows on (37 x 1001 x 777 7.8 against 12.4 us, 64 x 4096 x 512 6.7 against 13.8), either way at
//    16 (1024 x 1024 8.2 against 6.7, 1001 x 777 7.7 against 9.3) and wrong for one (1024 x 1024 8.3 against 5.5, 4096 x
//    512 6.5 against 5.8).  Beyond 8 blocks the rows kernel is worth two launches: 64 x 4096 x 4096 19.4 against 14.4, in
//    a graph 18.8 against 11.7.
inline bool direct_8bit(int m, int n, int k) {
    const int blocks = ceil_div(k, kBlock);
    if (m <= 64) return blocks <= 8;
    return blocks <= 16 || plan_matmul(m, n, k).splits == 1;
}

}  // namespace rs
