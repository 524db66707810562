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

}  // namespace rs
