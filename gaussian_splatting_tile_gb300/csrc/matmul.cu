// Matrix product of two 8-bit matrices with a scale for each block of 128 along the contracted axis.
//
// out[i][j] = sum_b sa[b][i] sb[b][j] sum_{t in block b} a[i][t] b[j][t]
//
// The inner sums are e4m3 products on the tensor cores (tcgen05.mma kind::f8f6f4, operands staged in shared memory by
// TMA, accumulators in tensor memory).  The scales change from block to block, so a block's 128 products are summed
// by themselves in tensor memory and then added, scaled, to a float32 total that stays in the registers of the
// threads that read it back: thread = row, so a's scale is one number a thread, and with a scale per 128 rows of b
// one number a warp -- one fused multiply-add per value and block.  (With a scale for every row of b a multiplication
// more.)
//
// What bounds it: 128 products take 256 x 256 outputs of two SMs about 490 clocks on the tensor cores; adding them up
// takes each of their schedulers 8192 multiply-adds, 390 clocks at the rate that two warps reach.  The two overlap,
// but each accumulator's way round (products, word to the readers, reading, word back) is longer than both, and there
// is room for two: that, and every instruction between the readers' loads, is what large products wait for.  Products
// with few blocks are bound by the results' way out. Measured: 65536 x 2048 x 2048 float16 out 240 us (2.3 PFLOP/s;
// without any adding up the same loads and products would take 148), 8192^3 2.6 PFLOP/s, 160,000 x 512 x 512 bf16 56
// us (4.4 TB/s; 37 at the copy's rate), dW of a layer (512 x 256 x 160,000, a scale a row) 45 us from a cold cache, 1
// x 4096 x 4096 9.5 us, as long as its call.  Rows of out that are not on 16-byte boundaries leave value by value: 160,000
// x 501 x 512 113 us from a cold cache where 512 columns take 88.
//
// An 8-bit result: with 256 columns a tile a reader holds a row's 128 sums of one block, so it settles the block's scale
// by itself, and a pass out is 128 bytes a row.  160,000 x 512 x 512 58 us (a float32 result and its 8-bit form: 181),
// bound by the readers: 40 for adding the blocks up, as above, and 18 for the way out, most of it the conversions (memory
// and products need 25 each).  Results by plain stores instead of TMA and the fence before it 66; loads of 32 columns
// from tensor memory, which do not fit the registers, 69.
#include <cuda.h>

#include <cfloat>

#include "wide.cuh"

namespace rs {
namespace {

__device__ unsigned int g_matmul_error;  // set when a bounded wait gave up

struct MatmulArgs {
    int m, n, k;
    const uint8_t* a; size_t as;
    const uint8_t* b; size_t bs;
    const float* sa;            // [blocks][m]
    const float* sb;            // [blocks][n], or [blocks][ceil(n / 128)]
    int relu;
    void* out; size_t os;
    int tma_cols;               // columns of out that TMA writes, a multiple of 16 bytes (0: none)
    int splits, tiles_n, tiles;
    int each, extra;            // blocks a stretch; the first `extra` stretches have one more
    float* part;                // splits > 1: [split][tile][column][128 rows]
    float* so;                  // out in 8 bits: its scales [ceil(n / 128)][m]
};

// ---------------------------------------------------------------- tensor cores, TMA, barriers
constexpr uint32_t kWaitPolls = 1u << 20;  // of at most a microsecond each

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Arrival at a barrier of another CTA of the cluster (address from cluster_addr).  It says that tensor memory has
// been read, nothing that this thread has stored: a release at the cluster's scope would wait for all of the thread's
// memory operations each time (measured: half the product's speed).
__device__ __forceinline__ void bar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// The address of `p`'s counterpart in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t addr, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok) : "r"(addr), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_wait(uint32_t addr, uint32_t parity) {
    if (bar_test(addr, parity)) return true;
    for (uint32_t i = 0; i < kWaitPolls; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok) : "r"(addr), "r"(parity) : "memory");
        if (ok) return true;
    }
    atomicOr(&g_matmul_error, 1u);
    return false;
}

__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity) { return bar_wait(smem_u32(b), parity); }

// A tile's corner (x: element along the row, y: row); x is a multiple of 128 bytes.
__device__ __forceinline__ void tma_load(const CUtensorMap* map, void* dst, uint64_t* bar, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}

// The same by one CTA of a pair, into its own memory, counted at a barrier of either (address from cluster_addr).
__device__ __forceinline__ void tma_load_pair(const CUtensorMap* map, void* dst, uint32_t bar, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// Matrix descriptor of a K-major operand in 128-byte swizzled rows (PTX ISA "Matrix Descriptors"): address >> 4,
// groups of eight rows 1024 bytes apart (bits 32-45), 0b001 at bits 46-48, 128-byte swizzle = 2 at bits 61-63.
__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr) {
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(64) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}

// Instruction descriptor of kind::f8f6f4 with e4m3 operands (type 0), both K-major, float32 sums.
template <int M, int N>
__host__ __device__ constexpr uint32_t tc_idesc() {
    return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// The same of a pair of CTAs: operands at the same places of both, the sums' upper 128 rows in the second's tensor
// memory.
__device__ __forceinline__ void tc_mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {  // arrives at both CTAs' barriers
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"(uint16_t(3)) : "memory");
}
// True in one lane of a converged warp.  The loops that feed the tensor cores run in all lanes and let one act: what
// they compute is then the same in every lane by construction, as those instructions' operands have to be.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of this warp's 32 lanes; the registers are valid after tc_wait.
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32"
                 " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));  // no use of them moves above the wait
}

__device__ __forceinline__ void copy4(float* dst, const float* src) {  // asynchronously
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Two floats in one register pair: a product or a multiply-add of both is one instruction (f32x2).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ---------------------------------------------------------------- the tile kernel
// A pair of CTAs takes 256 x BN tiles of out (and one of `splits` stretches of the blocks), persistently: each CTA
// holds 128 rows of a and half of b's rows, and one product instruction (cta_group::2) uses both, so that b is
// fetched and stored once a pair.  Warp 0 of each CTA loads, warp 1 of the first issues the products, warp 2 of each
// fetches the scales, warps 4 to 11 of both add the blocks up: warp w reads tensor-memory lanes 32 (w mod 4) on and a
// half of the columns. Tensor memory holds kAcc accumulators of BN columns: the products of the next blocks run while
// a block is read.
//
// What was tried and not kept (8192^3, each against the kernel of the time): single CTAs with 128 x 256 tiles, 476
// against 431 us; sixteen warps adding up 64 columns each, which do not fit the registers without moves, 527 against
// 420; accumulators of 128 columns, twice as many, 494 against 463 (160,000 x 512 x 512: 66 against 68); scalar
// multiply-adds instead of pairs, 472 against 459; the scales fetched by the readers themselves, a little better here
// (431) and worse where tiles are short (160,000 x 512 x 512: 76); asking for the next accumulator early, nothing.
constexpr int kSumWarps = 8;
constexpr int kTileThreads = 128 + 32 * kSumWarps;
// Registers a thread before and after the split between warps 0-3 and the rest: 128 x 40 + 256 x 232 = 384 x 168.  With a
// scale a row and 256 columns, and one a block and 128 columns, 20 bytes spill.
constexpr int kRegsLaunch = 168, kRegsFew = 40, kRegsMany = 232;
static_assert(128 * kRegsFew + 32 * kSumWarps * kRegsMany <= kTileThreads * kRegsLaunch, "the launch's registers");

template <int BN>
struct TileSmem {
    static constexpr int kStages = BN == 256 ? 4 : 6, kAcc = 512 / BN;
    uint8_t a[kStages][128 * 128];
    uint8_t b[kStages][BN / 2 * 128];
    uint8_t stage[kSumWarps][2][32 * 128];  // a warp's way out: twice 32 rows of 128 bytes
};
// A pair holds all of tensor memory of an SM while it waits for its other half to get the same.  No other pair may be in
// its way: two CTAs of them do not fit an SM's shared memory.  (Whatever else holds tensor memory frees it without waiting
// for another CTA.)
constexpr size_t kSmemSm = 228 * 1024;
static_assert(2 * sizeof(TileSmem<128>) > kSmemSm && 2 * sizeof(TileSmem<256>) > kSmemSm, "one pair's CTA an SM");

// The blocks of a stretch.  Between tiles every warp asks for them, so no division of 64 bits stands here, and unsplit
// products divide once for a tile: 160,000 x 512 x 512 bfloat16 out 66 -> 60 to 62 us, float32 out 91 -> 85.
struct Range { int first, last; };
__device__ __forceinline__ Range blocks_of(const MatmulArgs& g, int s) {
    const int first = s * g.each + min(s, g.extra);
    return {first, first + g.each + (s < g.extra ? 1 : 0)};
}
// Unit u is tile u mod tiles of stretch u / tiles.
struct Unit { int tile; Range r; };
__device__ __forceinline__ Unit unit_of(const MatmulArgs& g, int u) {
    const int s = g.splits > 1 ? u / g.tiles : 0;
    return {u - s * g.tiles, blocks_of(g, s)};
}

// max(x, 0), a NaN kept.
__device__ __forceinline__ float relu(float x) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
    return r;
}
// A warp's 32 rows x 128 bytes of results (thread = row, eight 16-byte words) in shared memory, the words of row r at
// word ^ (r mod 8): the 128-byte swizzle of the tensor map that takes them out, and no two of eight neighbours share
// a bank.
__device__ __forceinline__ void stage_rows(uint8_t* st, const uint4 (&w)[8], int lane) {
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(st + lane * 128 + ((i ^ (lane & 7)) << 4)) = w[i];
}
// From there to rows of out that TMA cannot write (not on 16-byte boundaries), one value a lane: two stores of 64
// bytes a row of 16-bit values.  (Words put together from neighbours, a store fewer, took 1.6 times as long.)
template <typename T>
__device__ __forceinline__ void copy_rows(const uint8_t* st, T* o, size_t os, long long rows, int cols, int lane) {
    constexpr int kPer = 16 / sizeof(T);
    const int n = int(min(rows, 32LL));
#pragma unroll 4
    for (int r = 0; r < n; ++r)
#pragma unroll
        for (int c = lane; c < 8 * kPer; c += 32)
            if (c < cols)
                o[r * os + c] =
                    *reinterpret_cast<const T*>(st + r * 128 + (((c / kPer) ^ (r & 7)) << 4) + c % kPer * sizeof(T));
}
// The last columns [first, cols) of this lane's row, fewer than 16 bytes, where the row ends inside these 128 bytes.
template <typename T>
__device__ __forceinline__ void copy_rest(const uint8_t* st, T* o, int first, int cols, int lane) {
    constexpr int kPer = 16 / sizeof(T);
    if (first < 0 || first >= 8 * kPer || first >= cols) return;
    const T* w = reinterpret_cast<const T*>(st + lane * 128 + (((first / kPer) ^ (lane & 7)) << 4));
    for (int c = first; c < cols; ++c) o[c] = w[c - first];
}
// TMA leaves out the box's columns past the tensor's only in whole words of 16 bytes: the map of out ends with the last
// whole word (tma_cols), and copy_rest writes what is left.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(x), "r"(y), "r"(smem_u32(src)) : "memory");
}

// ---- scales whose product is no normal float32
// With a scale per 128 rows of b the two scales are multiplied first, once for a row and block.  Where that leaves the
// normal numbers (below 2^-126 bits are lost, above 2^128 it is infinite) though the block's sum would bring the result
// back, the row's results are formed anew by its thread after the tiles, one scale after the other.  The warp that
// fetches the scales looks for such products before it overwrites them, which costs nothing: 160,000 x 512 x 512 56.0
// us back to back with it and without, 65536 x 2048 x 2048 224 and 225.  A warp of its own was 2 us slower a call where
// its code had to come from memory, a second way through the loop that adds the blocks up 10 to 20 percent on
// wide products, remembering there that such a product was met 3 to 5.
__device__ __forceinline__ bool normal(float f) { return fabsf(f) >= FLT_MIN && fabsf(f) <= FLT_MAX; }

// Whether some block of a stretch needs that: the product of its scales is not normal, and not only small because all of
// the row's values are zero (their scale is 2^-109: with small weights that is common, and the sum is zero either way).
__device__ __forceinline__ bool scales_apart(const MatmulArgs& g, Range r, long long row, int col) {
    const int per = (g.n + kBlock - 1) / kBlock;
#pragma unroll 1
    for (int b = r.first; b < r.last; ++b) {
        const float fa = g.sa[size_t(b) * g.m + row], fb = g.sb[size_t(b) * per + col / kBlock];
        if (normal(fa * fb) || fa == 0.f || fb == 0.f) continue;
        if (!(fabsf(fa * fb) < FLT_MIN)) return true;
        const uint8_t* a = g.a + row * g.as + size_t(b) * kBlock;
        const int len = min(kBlock, g.k - b * kBlock);
        uint32_t any = 0;
#pragma unroll
        for (int t = 0; t < kBlock; t += 16)
            if (t + 16 <= len) {
                const uint4 w = *reinterpret_cast<const uint4*>(a + t);
                any |= w.x | w.y | w.z | w.w;
            }
        for (int t = len & ~15; t < len; ++t) any |= a[t];
        if (any & 0x7f7f7f7fu) return true;
    }
    return false;
}

// Calls put(j, value) for this row's columns col + j, j < cols.
template <typename Put>
__device__ __forceinline__ void row_anew(const MatmulArgs& g, Range r, long long row, int col, int cols, Put&& put) {
    const int per = (g.n + kBlock - 1) / kBlock;
#pragma unroll 1
    for (int j = 0; j < cols && col + j < g.n; ++j) {
        float v = 0.f;
#pragma unroll 1
        for (int b = r.first; b < r.last; ++b) {
            const uint8_t* x = g.a + row * g.as + size_t(b) * kBlock;
            const uint8_t* y = g.b + (col + j) * g.bs + size_t(b) * kBlock;
            const int len = min(kBlock, g.k - b * kBlock);
            float sum = 0.f;
#pragma unroll 1
            for (int t = 0; t < len; ++t) {
                uint32_t xy;  // the two values as halves
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(xy) : "h"(uint16_t(x[t] | y[t] << 8)));
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&xy));
                sum = fmaf(f.x, f.y, sum);
            }
            v = fmaf(sum * g.sb[size_t(b) * per + (col + j) / kBlock], g.sa[size_t(b) * g.m + row], v);
        }
        put(j, v);
    }
}

// A thread's row and columns of the pair's tiles, where they need it.  Out of line: rarely called, and inlined it lies in
// the way of the code that always runs.
template <typename T, int BN>
__device__ __noinline__ void units_anew(const MatmulArgs& g, int pair, int pairs, int rank, int lane_row, int half) {
    constexpr int kCols = BN / (kSumWarps / 4);
    for (int u = pair; u < g.tiles * g.splits; u += pairs) {
        const auto [tile, r] = unit_of(g, u);
        const int ty = tile / g.tiles_n, col = (tile - ty * g.tiles_n) * BN + half * kCols;
        const long long row = (long long)(ty * 2 + rank) * 128 + lane_row;
        if (row >= g.m || col >= g.n || !scales_apart(g, r, row, col)) continue;
        T* out = static_cast<T*>(g.out) + row * g.os + col;
        if constexpr (sizeof(T) == 1) {  // the row's 128 columns twice: for their largest magnitude, and in 8 bits
            const auto value = [&](float x) { return g.relu ? relu(x) : x; };
            float top = 0.f, scale, inv;
            row_anew(g, r, row, col, kCols, [&](int, float x) { top = fmaxf(top, fabsf(value(x))); });
            block_scale(top, scale, inv);
            g.so[size_t(col / kBlock) * g.m + row] = scale;
            row_anew(g, r, row, col, kCols,
                     [&](int j, float x) { out[j] = uint8_t(e4m3x4(value(x) * inv, 0.f, 0.f, 0.f)); });
        } else {
            float* part = g.part + ((size_t(u) * 2 + rank) * BN + half * kCols) * 128 + lane_row;
            row_anew(g, r, row, col, kCols, [&](int j, float x) {
                if (g.splits > 1) part[size_t(j) * 128] = x;
                else out[j] = from_f<T>(g.relu ? relu(x) : x);
            });
        }
    }
}

template <typename T, int BN, bool ROWS>
__global__ void __launch_bounds__(kTileThreads, 1)
    k_matmul_tile(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_out, const __grid_constant__ MatmulArgs g) {
    RS_PDL_ENTER();
    using Smem = TileSmem<BN>;
    constexpr int kStages = Smem::kStages, kAcc = Smem::kAcc, kCols = BN / (kSumWarps / 4);
    extern __shared__ uint8_t raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[kAcc], acc_empty[kAcc];
    __shared__ uint32_t tmem_slot;
    // The scales of kRing blocks: a's of the CTA's rows, then b's of the tile's columns (ROWS) or of its halves.
    // Four blocks share a barrier, so that the readers ask and answer once in four.
    constexpr int kRing = 16, kGroups = kRing / 4, kScales = 128 + (ROWS ? BN : 4);
    __shared__ __align__(16) float scales[kRing][kScales];
    __shared__ uint64_t sc_full[kGroups], sc_empty[kGroups];
    __shared__ bool apart_met;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x & 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) bar_init(&full[i], 1), bar_init(&empty[i], 1);
        for (int i = 0; i < kAcc; ++i) bar_init(&acc_full[i], 1), bar_init(&acc_empty[i], 2 * kSumWarps);
        for (int i = 0; i < kGroups; ++i) bar_init(&sc_full[i], 32), bar_init(&sc_empty[i], kSumWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are set up before anything arrives there
    tc_after();
    const uint32_t tmem = tmem_slot;
    const int units = g.tiles * g.splits, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
        if (warp == 0) {
            const uint32_t bar0 = cluster_addr(full, 0);  // the first CTA's barriers count both CTAs' copies
            uint32_t s = 0, phase = 1, it = 0;
            bool ok = true;
            for (int u = pair; u < units && ok; u += pairs) {
                const auto [tile, r] = unit_of(g, u);
                const int ty = tile / g.tiles_n, y = (ty * 2 + rank) * 128,
                          x = (tile - ty * g.tiles_n) * BN + rank * (BN / 2);
                for (int b = r.first; b < r.last; ++b, ++it) {
                    if (!(ok = __all_sync(0xffffffffu, bar_wait(&empty[s], phase)))) break;
                    if (elect_one()) {
                        if (rank == 0) bar_expect(&full[s], 2 * (128 + BN / 2) * 128);
                        tma_load_pair(&map_a, sm.a[s], bar0 + s * 8, b * kBlock, y);
                        tma_load_pair(&map_b, sm.b[s], bar0 + s * 8, b * kBlock, x);
                    }
                    __syncwarp();
                    if (++s == kStages) s = 0, phase ^= 1;
                }
            }
            // no copy and no arrival may outlast the CTA: a stage's products follow its copies
            for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
                bar_wait(&empty[i % kStages], i / kStages & 1);
        } else if (warp == 1 && rank == 0) {
            const uint64_t da0 = tc_desc(smem_u32(sm.a[0])), db0 = tc_desc(smem_u32(sm.b[0]));
            uint32_t s = 0, phase = 0, h = 0, acc_phase = 1, it = 0;
            bool ok = true, ready = false;
            for (int u = pair; u < units && ok; u += pairs) {
                const Range r = unit_of(g, u).r;
                for (int b = r.first; b < r.last; ++b, ++it) {
                    ok = (ready || bar_wait(&full[s], phase)) && bar_wait(&acc_empty[h], acc_phase);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_after();
                    if (elect_one()) {
                        const uint64_t da = da0 + s * (sizeof(sm.a[0]) >> 4), db = db0 + s * (sizeof(sm.b[0]) >> 4);
                        const uint32_t d = tmem + h * BN;
#pragma unroll
                        for (int t = 0; t < 4; ++t)  // 32 bytes of K an instruction
                            tc_mma_pair(d, da + 2 * t, db + 2 * t, tc_idesc<256, BN>(), t > 0);
                        tc_commit_pair(&acc_full[h]);
                        tc_commit_pair(&empty[s]);
                    }
                    __syncwarp();
                    if (++s == kStages) s = 0, phase ^= 1;
                    if (++h == kAcc) h = 0, acc_phase ^= 1;
                    ready = __all_sync(0xffffffffu, bar_test(smem_u32(&full[s]), phase));  // while the products run
                }
            }
            if (!ok && it > 0) bar_wait(&acc_full[(it - 1) % kAcc], (it - 1) / kAcc & 1);  // products in flight
        } else if (warp == 2) {
            // The scales, up to kRing blocks ahead of their use and on into the next tiles: a load takes longer than
            // a block. Rows and columns outside the matrices take the last one's: what comes of them is not stored.
            const int per = ROWS ? g.n : (g.n + kBlock - 1) / kBlock;  // b's scales a block
            uint32_t count = 0;  // of blocks
            bool ok = true;
            const auto done = [&] {  // with the copies of a group, when they are
                const uint32_t bar = smem_u32(&sc_full[(count >> 2) % kGroups]);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
            };
            // Before scales are overwritten, and at the end: the largest and smallest magnitudes of four rows and of b's
            // two bound the products of a block.
            float least = 1.f, most = 1.f;
            const auto look = [&](uint32_t first, uint32_t last) {
#pragma unroll 1
                for (uint32_t i = first; i < last; ++i) {
                    const float4 v = reinterpret_cast<const float4*>(scales[i])[lane];
                    const float2 s = *reinterpret_cast<const float2*>(scales[i] + 128);
                    const float lo = fminf(fminf(fabsf(v.x), fabsf(v.y)), fminf(fabsf(v.z), fabsf(v.w)));
                    const float hi = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
                    least = fminf(least, lo * fminf(fabsf(s.x), fabsf(s.y)));
                    most = fmaxf(most, hi * fmaxf(fabsf(s.x), fabsf(s.y)));
                }
            };
            for (int u = pair; u < units && ok; u += pairs) {
                const auto [tile, r] = unit_of(g, u);
                const int ty = tile / g.tiles_n, x = (tile - ty * g.tiles_n) * BN;
                const long long y = (long long)(ty * 2 + rank) * 128 + lane;
                const float* pa = g.sa + size_t(r.first) * g.m;
                const float* pb = g.sb + size_t(r.first) * per;
                for (int b = r.first; b < r.last; ++b, pa += g.m, pb += per) {
                    if (count % 4 == 0) {
                        const uint32_t parity = (count / kRing & 1) ^ 1;
                        ok = __all_sync(0xffffffffu, bar_wait(&sc_empty[(count >> 2) % kGroups], parity));
                        if (!ok) break;
                        if (!ROWS && count >= kRing) {
                            look(count % kRing, count % kRing + 4);
                            __syncwarp();
                        }
                    }
                    float* to = scales[count % kRing];
#pragma unroll
                    for (int i = 0; i < 128; i += 32) copy4(to + i + lane, pa + min(y + i, (long long)g.m - 1));
                    if (ROWS) {
#pragma unroll
                        for (int i = 0; i < BN; i += 32) copy4(to + 128 + i + lane, pb + min(x + i + lane, per - 1));
                    } else if (lane < 2) {
                        copy4(to + 128 + lane, pb + min((x + lane * kCols) / kBlock, per - 1));
                    }
                    if (count % 4 == 3) done();
                    ++count;
                }
            }
            if (count % 4 != 0) done();
            asm volatile("cp.async.wait_all;" ::: "memory");
            if constexpr (!ROWS) {
                __syncwarp();  // the other lanes' copies
                look(0, min(count, uint32_t(kRing)));
                const bool met = __any_sync(0xffffffffu, !(least >= FLT_MIN && most <= FLT_MAX));
                if (lane == 0) apart_met = met;
                __syncwarp();
                asm volatile("bar.arrive 1, %0;" ::"n"(32 + 32 * kSumWarps) : "memory");
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        const int w8 = warp - 4, half = w8 >> 2, wrow = (w8 & 3) * 32;   // columns and rows of the tile
        const uint32_t lanes = tmem + (uint32_t(wrow) << 16) + half * kCols;
        const uint32_t full0 = smem_u32(acc_full), empty0 = cluster_addr(acc_empty, 0);
        const uint32_t sc_full0 = smem_u32(sc_full), sc_empty0 = smem_u32(sc_empty);
        uint32_t h = 0, phase = 0;         // the accumulator to read next
        uint32_t count = 0;                // of blocks
        bool ok = true;
        for (int u = pair; u < units; u += pairs) {
            const auto [tile, r] = unit_of(g, u);
            const int ty = tile / g.tiles_n;
            const long long row0 = (long long)(ty * 2 + rank) * 128 + wrow;
            const int col = (tile - ty * g.tiles_n) * BN + half * kCols;
            uint64_t acc[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) acc[j] = 0;
            for (int b = r.first; b < r.last; ++b) {
                const uint32_t group = (count >> 2) % kGroups;
                // a wait that gave up ends the waiting, not the loop: what is added from then on is not stored
                if (count % 4 == 0)
                    ok = ok && bar_wait(sc_full0 + group * 8, count / kRing & 1);
                const float* sc = scales[count % kRing];
                const float* sb = sc + 128 + (ROWS ? half * kCols : half);
                const float f = ROWS ? sc[wrow + lane] : sc[wrow + lane] * sb[0];
                const uint64_t ff = pack2(f, f);
                if (!ROWS && count % 4 == 3) {
                    __syncwarp();
                    if (lane == 0) bar_arrive(sc_empty0 + group * 8);
                }
                ok = ok && bar_wait(full0 + h * 8, phase);
                __syncwarp();
                tc_after();
                uint32_t v[2][16];
                tc_ld16(lanes + h * BN, v[0]);
#pragma unroll
                for (int c = 0; c < kCols / 16; ++c) {
                    tc_wait(v[c & 1]);
                    if (c + 1 < kCols / 16) {
                        tc_ld16(lanes + h * BN + 16 * (c + 1), v[(c + 1) & 1]);
                    } else {  // all of it has been read
                        tc_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive_cluster(empty0 + h * 8);
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        uint64_t p = pack2(v[c & 1][j], v[c & 1][j + 1]), q = pack2(v[c & 1][j + 2], v[c & 1][j + 3]);
                        if (ROWS) {
                            const ulonglong2 s4 = *reinterpret_cast<const ulonglong2*>(sb + 16 * c + j);
                            p = mul2(p, s4.x);
                            q = mul2(q, s4.y);
                        }
                        acc[8 * c + j / 2] = fma2(p, ff, acc[8 * c + j / 2]);
                        acc[8 * c + j / 2 + 1] = fma2(q, ff, acc[8 * c + j / 2 + 1]);
                    }
                }
                if (ROWS && count % 4 == 3) {
                    __syncwarp();
                    if (lane == 0) bar_arrive(sc_empty0 + group * 8);
                }
                ++count;
                if (++h == kAcc) h = 0, phase ^= 1;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (sizeof(T) > 1 && g.splits > 1) {
                float* o = g.part + ((size_t(u) * 2 + rank) * BN + half * kCols) * 128 + wrow + lane;
#pragma unroll
                for (int j = 0; j < kCols / 2; ++j) {
                    const float2 x = unpack2(acc[j]);
                    o[size_t(2 * j) * 128] = x.x;
                    o[size_t(2 * j + 1) * 128] = x.y;
                }
            } else if (col < g.n) {
                // Passes of 128 bytes a row, two to a fence (half of the way out's time was the fence).
                // In 8 bits a pass is a block: its scale is settled in the thread that holds the row's 128 sums.
                constexpr int kOnce = 128 / sizeof(T), kPasses = kCols / kOnce, kTogether = kPasses < 2 ? kPasses : 2;
                float inv = 1.f;
                if constexpr (sizeof(T) == 1) {
                    static_assert(kCols == kBlock, "a thread's columns are one block");
                    float top = 0.f, scale;
                    if (g.relu) {  // which the conversion does, too
#pragma unroll
                        for (int j = 0; j < kCols / 2; ++j) top = max3(top, unpack2(acc[j]).x, unpack2(acc[j]).y);
                    } else {
#pragma unroll
                        for (int j = 0; j < kCols / 2; ++j)
                            top = max3(top, fabsf(unpack2(acc[j]).x), fabsf(unpack2(acc[j]).y));
                    }
                    block_scale(top, scale, inv);
                    if (row0 + lane < g.m) g.so[size_t(col / kBlock) * g.m + row0 + lane] = scale;
                }
#pragma unroll
                for (int c = 0; c < kPasses; c += kTogether) {
                    // what was copied out of the buffers before has left them
                    if (g.tma_cols && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < kTogether; ++q) {
                        uint4 w[8];
                        uint32_t* ww = reinterpret_cast<uint32_t*>(w);
                        if constexpr (sizeof(T) == 1) {
                            const uint64_t by = pack2(inv, inv);
#pragma unroll
                            for (int j = 0; j < kOnce / 2; ++j) acc[j] = mul2(acc[j], by);
                            const auto words = [&](auto convert) {
#pragma unroll
                                for (int j = 0; j < kOnce; j += 4) {
                                    const float2 x = unpack2(acc[j / 2]), y = unpack2(acc[j / 2 + 1]);
                                    ww[j / 4] = convert(x.x, x.y, y.x, y.y);
                                }
                            };
                            if (g.relu) words([](float a, float b, float c, float d) { return e4m3x4<true>(a, b, c, d); });
                            else words([](float a, float b, float c, float d) { return e4m3x4(a, b, c, d); });
                        } else
#pragma unroll
                        for (int j = 0; j < kOnce; j += 2) {
                            float2 x = unpack2(acc[((c + q) * kOnce + j) / 2]);
                            if (g.relu) x = make_float2(relu(x.x), relu(x.y));
                            if constexpr (sizeof(T) == 4) {
                                ww[j] = __float_as_uint(x.x);
                                ww[j + 1] = __float_as_uint(x.y);
                            } else {
                                ww[j / 2] = pack_pair(x.x, x.y, T());
                            }
                        }
                        stage_rows(sm.stage[w8][q], w, lane);
                    }
                    if (g.tma_cols) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < kTogether; ++q) {
                        const int x = col + (c + q) * kOnce;
                        if (!g.tma_cols) {
                            copy_rows(sm.stage[w8][q], static_cast<T*>(g.out) + row0 * g.os + x, g.os, g.m - row0,
                                      g.n - x, lane);
                        } else {
                            if (lane == 0 && row0 < g.m && x < g.tma_cols)
                                tma_store(&map_out, sm.stage[w8][q], x, int(row0));
                            if (row0 + lane < g.m)
                                copy_rest(sm.stage[w8][q], static_cast<T*>(g.out) + (row0 + lane) * g.os + x,
                                          g.tma_cols - x, g.n - x, lane);
                        }
                    }
                    if (g.tma_cols && lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // no copy outlasts the CTA
        __syncwarp();
        if constexpr (!ROWS) {
            asm volatile("bar.sync 1, %0;" ::"n"(32 + 32 * kSumWarps) : "memory");
            if (ok && apart_met) units_anew<T, BN>(g, pair, pairs, rank, wrow + lane, half);
            __syncwarp();
        }
    }
    tc_before();
    __syncthreads();
    cluster_sync();  // neither CTA's memory goes while the other's products or arrivals use it
    tc_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ---------------------------------------------------------------- few rows
// With at most 64 rows of a the time goes into reading b once, so the roles change sides: the products' 128 rows are
// rows of b (weights), their NT columns the rows of a, and a cluster of up to 8 CTAs shares a tile's blocks: all
// SMs read from 18 tiles on, 2305 rows of b.  Each CTA adds its blocks up as the tile kernel does (thread = row of b); the cluster then adds its
// CTAs' sums through distributed shared memory, rank by rank, each CTA finishing some of the columns.
constexpr int kRowsTmem = 128;  // columns of tensor memory

template <int NT>
struct RowsSmem {
    static constexpr int kStage = 128 * 128 + NT * 128, kAcc = kRowsTmem / NT, kMaxStages = 8;
};

template <typename T, int NT, bool ROWS>
__global__ void __launch_bounds__(192)
    k_matmul_rows(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, MatmulArgs g,
                  int stages) {
    RS_PDL_ENTER();
    constexpr int kStage = RowsSmem<NT>::kStage, kAcc = RowsSmem<NT>::kAcc, kMax = RowsSmem<NT>::kMaxStages;
    extern __shared__ uint8_t raw[];
    uint8_t* ops = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kMax], empty[kMax], acc_full[kAcc], acc_empty[kAcc];
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float sbuf[4][2][NT];  // a warp's copy of a's scales of one block
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % g.splits, tile = blockIdx.x / g.splits, n0 = tile * 128;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) bar_init(&full[i], 1), bar_init(&empty[i], 1);
        for (int i = 0; i < kAcc; ++i) bar_init(&acc_full[i], 1), bar_init(&acc_empty[i], 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(kRowsTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_slot;
    const Range r = blocks_of(g, rank);
    const int count = r.last - r.first;
    const int wrow = (warp & 3) * 32 + lane;
    float acc[NT];
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (; it < count; ++it) {
                const int s = it % stages;
                if (!(ok = bar_wait(&empty[s], (it / stages & 1) ^ 1))) break;
                bar_expect(&full[s], kStage);
                tma_load(&map_b, ops + s * kStage, &full[s], (r.first + it) * kBlock, n0);
                tma_load(&map_a, ops + s * kStage + 128 * 128, &full[s], (r.first + it) * kBlock, 0);
            }
            for (int i = max(0, it - stages); i < it; ++i)  // no copy and no arrival may outlast the CTA
                bar_wait(ok ? &empty[i % stages] : &full[i % stages], i / stages & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0;
            for (; it < count; ++it) {
                const int s = it % stages, h = it % kAcc;
                if (!(ok = bar_wait(&full[s], it / stages & 1) && bar_wait(&acc_empty[h], (it / kAcc & 1) ^ 1))) break;
                tc_after();
                const uint32_t at = smem_u32(ops + s * kStage);
                const uint64_t da = tc_desc(at), db = tc_desc(at + 128 * 128);
#pragma unroll
                for (int t = 0; t < 4; ++t) tc_mma(tmem + h * NT, da + 2 * t, db + 2 * t, tc_idesc<128, NT>(), t > 0);
                tc_commit(&empty[s]);
                tc_commit(&acc_full[h]);
            }
            if (!ok && it > 0) bar_wait(&acc_full[(it - 1) % kAcc], (it - 1) / kAcc & 1);  // products in flight
        }
        __syncwarp();
    } else {
        const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
        const int per = ROWS ? g.n : (g.n + kBlock - 1) / kBlock, sc = ROWS ? n0 + wrow : tile;
        constexpr int kSa = (NT + 31) / 32;
        float nb = 0.f, na[kSa];
        auto load_scales = [&](int b) {
            nb = sc < per ? g.sb[size_t(b) * per + sc] : 0.f;
#pragma unroll
            for (int i = 0; i < kSa; ++i) na[i] = 32 * i + lane < g.m ? g.sa[size_t(b) * g.m + 32 * i + lane] : 0.f;
        };
        if (count > 0) load_scales(r.first);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = 0.f;
        for (int it = 0; it < count; ++it) {
            const int h = it % kAcc;
            const float f = nb;
            float* sa = sbuf[warp - 2][it & 1];
#pragma unroll
            for (int i = 0; i < kSa; ++i)
                if (32 * i + lane < NT) sa[32 * i + lane] = na[i];
            __syncwarp();
            if (it + 1 < count) load_scales(r.first + it + 1);
            ok = __all_sync(0xffffffffu, bar_wait(&acc_full[h], it / kAcc & 1));
            if (!ok) break;
            tc_after();
#pragma unroll
            for (int c = 0; c < NT / 16; ++c) {
                uint32_t v[16];
                tc_ld16(lanes + h * NT + 16 * c, v);
                tc_wait(v);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    acc[16 * c + j] = fmaf(__uint_as_float(v[j]) * sa[16 * c + j], f, acc[16 * c + j]);
            }
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(smem_u32(&acc_empty[h]));
        }
    }
    const int n = n0 + wrow;
    auto store = [&](int j, float v) {
        if (g.relu) v = relu(v);
        static_cast<T*>(g.out)[size_t(j) * g.os + n] = from_f<T>(v);
    };
    // Every role is done with the operands' memory and with tensor memory after this barrier.  The sums take the former's
    // place; the latter goes back before the first wait for the cluster, whose other CTAs may still be asking for theirs
    // on SMs where such CTAs of other launches hold it.
    tc_before();
    const bool all = __syncthreads_and(ok);
    tc_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kRowsTmem) : "memory");
    if (g.splits == 1) {
        if (warp >= 2 && all && n < g.n) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (j < g.m) store(j, acc[j]);
        }
    } else {
        float* red = reinterpret_cast<float*>(ops);
        if (warp >= 2) {
#pragma unroll
            for (int j = 0; j < NT; ++j) red[j * 128 + wrow] = all ? acc[j] : __int_as_float(0x7fc00000);
        }
        cluster_sync();
        if (warp >= 2 && n < g.n) {
            for (int j = rank; j < g.m; j += g.splits) {
                float v = 0.f;
                for (int s = 0; s < g.splits; ++s) {
                    float x;
                    const uint32_t there = cluster_addr(red + j * 128 + wrow, s);
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(there) : "memory");
                    v += x;
                }
                store(j, v);
            }
        }
        cluster_sync();  // no CTA's memory goes while another reads it
    }
}

// out from the partial sums of `splits` stretches. A block takes 8 columns of a tile, each of its GROUPS groups of
// eight warps every GROUPS-th stretch: a warp reads a column's 128 rows, eight stretches in flight; the groups' sums
// are added in order (the same every time), and the values leave through shared memory along out's rows.  What bounds
// it is the time of its loads, one after another. Four groups from ten stretches on, one below, where three would be
// idle and tiles many: the whole product at 76 stretches (128 x 64 x 160000) 27 us against 44 with one, at 19 (512 x
// 256 x 160000) 46 against 50, at 10 (1792 x 256 x 40000) 42 against 44, at 9 (512 x 256 x 9300) 19 against 17, at 3
// (2000 x 700 x 10000) 40 against 31.
constexpr int kManySplits = 10;
template <typename T, int GROUPS>
__global__ void __launch_bounds__(256 * GROUPS) k_matmul_join(MatmulArgs g, int bn) {
    RS_PDL_ENTER();
    constexpr int kAtOnce = 8;
    __shared__ __align__(16) float sm[GROUPS][8][132];  // 132: the reads of 8 columns x 4 rows hit different banks
    const int groups = bn / 8, half = blockIdx.x / groups, tile = half >> 1, c0 = blockIdx.x % groups * 8;
    const int lane = threadIdx.x & 31, cc = threadIdx.x >> 5 & 7, group = threadIdx.x >> 8;
    const float* p = g.part + (size_t(half) * bn + c0 + cc) * 128 + lane * 4;
    const size_t step = size_t(g.tiles) * 2 * bn * 128;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = group; s < g.splits; s += GROUPS * kAtOnce) {
        float4 w[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int at = s + i * GROUPS;
            w[i] = at < g.splits ? *reinterpret_cast<const float4*>(p + at * step) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) v.x += w[i].x, v.y += w[i].y, v.z += w[i].z, v.w += w[i].w;
    }
    *reinterpret_cast<float4*>(&sm[group][cc][lane * 4]) = v;
    __syncthreads();
    const int c = threadIdx.x & 7;
    const long long col = (long long)(tile % g.tiles_n) * bn + c0 + c;
#pragma unroll
    for (int i = 0; i < 128; i += 32 * GROUPS) {
        const int r = i + int(threadIdx.x >> 3);
        const long long row = (long long)(tile / g.tiles_n * 2 + (half & 1)) * 128 + r;
        float x = sm[0][c][r];
#pragma unroll
        for (int j = 1; j < GROUPS; ++j) x += sm[j][c][r];
        if (row < g.m && col < g.n) static_cast<T*>(g.out)[row * g.os + col] = from_f<T>(g.relu ? relu(x) : x);
    }
}

// ---------------------------------------------------------------- host side
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);
EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const char* name = "cuTensorMapEncodeTiled";
        const cudaError_t e = cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess) p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// A [rows][cols] matrix, moved in boxes of 128 bytes of a row and `box` rows; what lies outside reads as zero and is
// not written.
bool encode(CUtensorMap* map, CUtensorMapDataType type, size_t size, const void* p, size_t stride, int rows, int cols,
            int box) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)}, strides[1] = {cuuint64_t(stride * size)};
    const cuuint32_t boxes[2] = {cuuint32_t(128 / size), cuuint32_t(box)}, steps[2] = {1, 1};
    return f(map, type, 2, const_cast<void*>(p), dims, strides, boxes, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// With programmatic stream serialization, in clusters of `cluster` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), int cluster, unsigned grid, unsigned block, int smem,
                            cudaStream_t s, Args&&... args) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename T, int BN, bool ROWS>
cudaError_t launch_tile(const CUtensorMap& a, const CUtensorMap& b, const MatmulArgs& g, cudaStream_t s) {
    CUtensorMap out{};
    constexpr CUtensorMapDataType type = sizeof(T) == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (g.tma_cols && g.splits == 1 && !encode(&out, type, sizeof(T), g.out, g.os, g.m, g.tma_cols, 32))
        return cudaErrorUnknown;
    constexpr int smem = sizeof(TileSmem<BN>) + 1024;  // + room to align the base to 1 KB
    // the kernel's register split counts on what it is launched with
    static const bool enough = [] {
        cudaFuncAttributes f{};
        return cudaFuncGetAttributes(&f, k_matmul_tile<T, BN, ROWS>) == cudaSuccess && f.numRegs >= kRegsLaunch;
    }();
    if (!enough) return cudaErrorInvalidConfiguration;
    const unsigned grid = 2u * std::min(kPairs, g.tiles * g.splits);
    return launch_clusters(k_matmul_tile<T, BN, ROWS>, 2, grid, kTileThreads, smem, s, a, b, out, g);
}

template <typename T, int NT, bool ROWS>
cudaError_t launch_rows(const CUtensorMap& a, const CUtensorMap& b, const MatmulArgs& g, cudaStream_t s) {
    using Smem = RowsSmem<NT>;
    const int per = ceil_div(ceil_div(g.k, kBlock), g.splits), stages = std::min(per, Smem::kMaxStages);
    const int smem = std::max(stages * Smem::kStage, NT * 128 * 4) + 1024;
    const unsigned grid = unsigned(g.tiles) * g.splits;
    return launch_clusters(k_matmul_rows<T, NT, ROWS>, g.splits, grid, 192, smem, s, a, b, g, stages);
}

// 8-bit zeros have their scale too.
__global__ void k_zero_scales(float* scales, size_t n) {
    RS_PDL_ENTER();
    float scale, inv;
    block_scale(0.f, scale, inv);
    for (size_t i = blockIdx.x * size_t(blockDim.x) + threadIdx.x; i < n; i += size_t(gridDim.x) * blockDim.x)
        scales[i] = scale;
}

// The float32 result on its way to 8 bits, where the tile kernel does not write them itself: [m][n to 16 bytes].
size_t wide_row(int32_t n) { return (size_t(n) + 3) / 4 * 4; }
size_t wide_bytes(int32_t m, int32_t n) { return size_t(m) * wide_row(n) * sizeof(float); }

}  // namespace

int take_matmul_error() {
    unsigned int v = 0u;
    if (cudaMemcpyFromSymbol(&v, g_matmul_error, sizeof(v)) != cudaSuccess) return -1;
    if (v == 0u) return 0;
    const unsigned int zero = 0u;
    if (cudaMemcpyToSymbol(g_matmul_error, &zero, sizeof(zero)) != cudaSuccess) return -1;
    return 1;
}

}  // namespace rs

extern "C" {

size_t rs_matmul_fp8_workspace_size(int32_t m, int32_t n, int32_t k) {
    return m <= 0 || n <= 0 || k <= 0 ? 0 : rs::plan_matmul(m, n, k).workspace();
}

int rs_matmul_fp8(int32_t m, int32_t n, int32_t k, const uint8_t* d_a, size_t a_stride, const float* d_a_scales,
                  const uint8_t* d_b, size_t b_stride, const float* d_b_scales, int32_t b_scale_rows, int32_t relu,
                  int32_t out_dtype, void* d_out, size_t out_stride, void* d_workspace, size_t workspace_bytes,
                  void* stream) {
    using namespace rs;
    if (m < 0 || n < 0 || k < 0 || !dtype_ok(out_dtype) || (b_scale_rows != 1 && b_scale_rows != kBlock))
        return RS_ERR_INVALID_ARG;
    constexpr int32_t kMost = 0x7ffffc00;  // the last tile's rows still are numbers of 32 bits
    if (m > kMost || n > kMost || k > kMost) return RS_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return RS_OK;
    const size_t z = dtype_size(out_dtype);
    if (!ptr_ok(d_out, z) || out_stride < size_t(n)) return RS_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k == 0)
        return cudaMemset2DAsync(d_out, out_stride * z, 0, n * z, m, s) == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    if (!fp8_rows_ok(d_a, a_stride, k) || !fp8_rows_ok(d_b, b_stride, k) || !ptr_ok(d_a_scales, 4) ||
        !ptr_ok(d_b_scales, 4) || a_stride >= (size_t(1) << 40) || b_stride >= (size_t(1) << 40))
        return RS_ERR_INVALID_ARG;
    if ((long long)ceil_div(m, 128) * ceil_div(n, 128) > 0x3fffffff) return RS_ERR_INVALID_ARG;
    const Plan p = plan_matmul(m, n, k);
    const size_t need = p.workspace();
    if (need > 0 && !ptr_ok(d_workspace, 16)) return RS_ERR_INVALID_ARG;
    if (workspace_bytes < need) return RS_ERR_WORKSPACE;
    CUtensorMap ma, mb;
    constexpr CUtensorMapDataType bytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!encode(&ma, bytes, 1, d_a, a_stride, m, k, p.rows ? p.rows : 128) ||
        !encode(&mb, bytes, 1, d_b, b_stride, n, k, p.rows ? 128 : p.bn / 2))
        return RS_ERR_CUDA;
    const int blocks = ceil_div(k, kBlock);
    const int whole = n / int(16 / z) * int(16 / z);  // columns in whole words of 16 bytes
    const int tma_cols = rows16(d_out, out_stride, z) && out_stride * z < (size_t(1) << 40) ? whole : 0;
    MatmulArgs g{m, n, k, d_a, a_stride, d_b, b_stride, d_a_scales, d_b_scales, relu, d_out, out_stride, tma_cols,
                 p.splits, p.tiles_n, p.tiles, blocks / p.splits, blocks % p.splits, static_cast<float*>(d_workspace), nullptr};
    cudaError_t e = with_dtype(out_dtype, [&](auto v) {
        using T = decltype(v);
        const bool per_row = b_scale_rows == 1;
        const auto launch = [&](auto rows, auto blocks) { return per_row ? rows(ma, mb, g, s) : blocks(ma, mb, g, s); };
        if (p.rows == 16) return launch(launch_rows<T, 16, true>, launch_rows<T, 16, false>);
        if (p.rows == 32) return launch(launch_rows<T, 32, true>, launch_rows<T, 32, false>);
        if (p.rows == 64) return launch(launch_rows<T, 64, true>, launch_rows<T, 64, false>);
        if (p.bn == 256)
            return launch(launch_tile<T, 256, true>, launch_tile<T, 256, false>);
        return launch(launch_tile<T, 128, true>, launch_tile<T, 128, false>);
    });
    if (e == cudaSuccess && need > 0)
        e = with_dtype(out_dtype, [&](auto v) {
            using T = decltype(v);
            const bool many = p.splits >= kManySplits;
            return pdl_launch(many ? k_matmul_join<T, 4> : k_matmul_join<T, 1>, unsigned(p.tiles) * 2 * (p.bn / 8),
                              many ? 1024 : 256, 0, s, g, p.bn);
        });
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

size_t rs_matmul_fp8_q_workspace_size(int32_t m, int32_t n, int32_t k) {
    using namespace rs;
    if (m <= 0 || n <= 0 || k <= 0 || direct_8bit(m, n, k)) return 0;
    return wide_bytes(m, n) + (rs_matmul_fp8_workspace_size(m, n, k) + 15) / 16 * 16;
}

int rs_matmul_fp8_q(int32_t m, int32_t n, int32_t k, const uint8_t* d_a, size_t a_stride, const float* d_a_scales,
                    const uint8_t* d_b, size_t b_stride, const float* d_b_scales, int32_t b_scale_rows, int32_t relu,
                    uint8_t* d_q, size_t q_stride, float* d_scales, void* d_workspace, size_t workspace_bytes,
                    void* stream) {
    using namespace rs;
    if (m < 0 || n < 0 || k < 0 || (b_scale_rows != 1 && b_scale_rows != kBlock)) return RS_ERR_INVALID_ARG;
    constexpr int32_t kMost = 0x7ffffc00;
    if (m > kMost || n > kMost || k > kMost) return RS_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return RS_OK;
    if (!fp8_rows_ok(d_q, q_stride, n) || !ptr_ok(d_scales, 4) || q_stride >= (size_t(1) << 40))
        return RS_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k == 0) {
        const size_t count = size_t(ceil_div(n, kBlock)) * m;
        cudaError_t e = cudaMemset2DAsync(d_q, q_stride, 0, n, m, s);
        if (e == cudaSuccess)
            e = pdl_launch(k_zero_scales, unsigned(std::min<size_t>(ceil_div(count, 256), 8 * kSms)), 256, 0, s, d_scales,
                           count);
        return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    }
    if (!fp8_rows_ok(d_a, a_stride, k) || !fp8_rows_ok(d_b, b_stride, k) || !ptr_ok(d_a_scales, 4) ||
        !ptr_ok(d_b_scales, 4) || a_stride >= (size_t(1) << 40) || b_stride >= (size_t(1) << 40))
        return RS_ERR_INVALID_ARG;
    if ((long long)ceil_div(m, 128) * ceil_div(n, 128) > 0x3fffffff) return RS_ERR_INVALID_ARG;
    const size_t need = rs_matmul_fp8_q_workspace_size(m, n, k);
    if (need > 0 && !ptr_ok(d_workspace, 16)) return RS_ERR_INVALID_ARG;
    if (workspace_bytes < need) return RS_ERR_WORKSPACE;
    if (need > 0) {
        const size_t row = wide_row(n), first = wide_bytes(m, n);
        float* wide = static_cast<float*>(d_workspace);
        const int e = rs_matmul_fp8(m, n, k, d_a, a_stride, d_a_scales, d_b, b_stride, d_b_scales, b_scale_rows, relu,
                                    RS_F32, wide, row, static_cast<char*>(d_workspace) + first, workspace_bytes - first,
                                    stream);
        return e != RS_OK ? e
                          : rs_quantize_fp8(m, n, RS_F32, wide, row, nullptr, 0, d_q, q_stride, d_scales, nullptr, 0,
                                            nullptr, stream);
    }
    CUtensorMap ma, mb;
    constexpr CUtensorMapDataType bytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!encode(&ma, bytes, 1, d_a, a_stride, m, k, 128) || !encode(&mb, bytes, 1, d_b, b_stride, n, k, 128))
        return RS_ERR_CUDA;
    const int blocks = ceil_div(k, kBlock), tiles_n = ceil_div(n, 256), tiles = ceil_div(m, 256) * tiles_n;
    const MatmulArgs g{m, n, k, d_a, a_stride, d_b, b_stride, d_a_scales, d_b_scales, relu, d_q, q_stride, n / 16 * 16, 1,
                       tiles_n, tiles, blocks, 0, nullptr, d_scales};
    const cudaError_t e = b_scale_rows == 1 ? launch_tile<uint8_t, 256, true>(ma, mb, g, s)
                                            : launch_tile<uint8_t, 256, false>(ma, mb, g, s);
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
