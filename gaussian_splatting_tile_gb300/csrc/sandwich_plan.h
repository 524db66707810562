// How the sandwich norm's backward gives rows to threads and blocks, from its sizes alone.  Plain C++, so that a host compiler
// takes it by itself (the tests ask it how many rows a thread adds up).
#pragma once

#include "matmul_plan.h"

namespace rs {

// Threads of a block whose rows are `tpr` threads each: as many rows as 128 hold, one at least.
constexpr int block_threads(int tpr) { return tpr < 128 ? 128 / tpr * tpr : tpr; }
template <int TPR>
constexpr int kBlockThreads = block_threads(TPR);

// Threads of a row in a CTA and runs of eight values of each.  Two runs a thread; in 16 bits, for widths that would leave
// a quarter of those idle or more, one run on three quarters of the threads instead (100,000 x 768 bf16 from checkpoints
// on 96 threads 194 us, on 64 with two runs 237; float32 as stored 456, 362 with two).
struct Shape { int threads, runs; };
inline Shape bwd_shape(int cols, bool f32) {
    const int runs = ceil_div(cols, 8);
    if (runs <= 16) return {16, 1};
    if (runs <= 32) return {16, 2};
    if (runs <= 64) return {32, 2};
    if (runs <= 96 && !f32) return {96, 1};
    if (runs <= 128) return {64, 2};
    if (runs <= 192 && !f32) return {192, 1};
    if (runs <= 256) return {128, 2};
    if (runs <= 384 && !f32) return {384, 1};
    return {256, 2};
}
// CTAs of a row: a cluster from 4097 columns on.
inline int bwd_ctas(int cols) { return cols <= 4096 ? 1 : cols <= 8192 ? 2 : 4; }
// Blocks on an SM: registers.
constexpr int bwd_resident(int threads, int runs) { return runs == 1 ? 384 / threads : threads > 128 ? 1 : 2; }
// Rows that a block takes at once, and blocks (clusters) of a call, each with a row of partial sums, on a GPU that holds
// as many clusters as it has SMs for.
inline int bwd_rows(int cols, bool f32) {
    const Shape p = bwd_shape(cols, f32);
    return block_threads(p.threads) / p.threads;
}
inline int bwd_blocks(int rows, int cols, bool f32) {
    const Shape p = bwd_shape(cols, f32);
    const int most = kSms * bwd_resident(block_threads(p.threads), p.runs) / bwd_ctas(cols);
    return std::min(ceil_div(rows, bwd_rows(cols, f32)), most);
}

}  // namespace rs
