#include "sandwich.cuh"

namespace rs {
namespace {

// ---------------------------------------------------------------- backward
// The copies of a row's operands on their way.  Of rows on 16-byte boundaries every thread copies its own runs into a
// place of its own and reads them back itself, so the ring needs no barrier.  One or two rows are in flight for each that
// is worked on: two stages, or three where a stage is at most 24 KB.  Through L1, where the two halves of a float32 run's
// sectors meet (160,000 x 512 float32: 382 against 626 us past it).
//
// With `bytes`, that many of SIZE are read and the rest becomes zero.
template <int SIZE>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                 ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src), "n"(SIZE) : "memory");
}
template <int SIZE>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;"
                 ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src), "n"(SIZE), "r"(bytes) : "memory");
}

// Rows that are not on 16-byte boundaries come in words, neighbours' words by neighbouring threads: a warp's (a row's
// sixteen threads') runs follow each other in memory, so their words do, and one more where 16-bit runs start in the
// middle of a word.  A thread's run then was copied by others of its warp, so the warp meets before it copies over a stage
// and before it reads one.  (80,000 x 1001 bf16 as stored 382 us, float32 655; each thread its own run's words 434 and
// 894.)
template <typename T, bool KEPT, Move MOVE, int TPR, int RUNS>
struct Ring {
    static constexpr bool kWhole = MOVE != kAny;                               // runs on 16-byte boundaries
    static constexpr int kThreads = kBlockThreads<TPR>;
    static constexpr int kGroup = TPR < 32 ? TPR : 32, kGroups = kThreads / kGroup;
    static constexpr int kWords = kWhole ? int(sizeof(T)) / 2 : 2 * int(sizeof(T));  // a thread's: of 16 bytes, or of 4
    static constexpr int kGroupBytes = kGroup * (kWhole ? 16 : 4) * kWords + (kWhole || sizeof(T) == 4 ? 0 : 16);
    static constexpr int kWide = (KEPT ? 2 : 5) * RUNS, kNarrow = KEPT ? 3 * RUNS : 0;  // runs of T, of bytes
    static constexpr int kStage = kWide * kGroups * kGroupBytes + kNarrow * kThreads * 8;
    static constexpr int kStages = kStage <= 24 * 1024 ? 3 : 2;
    static constexpr int kBytes = kStages * kStage;
    static constexpr int kVectors = 3 * RUNS * TPR * 32;                       // behind the ring
    static constexpr int kShared = kBytes + kVectors;                          // what a block is launched with
    static_assert((kThreads == TPR || kBytes >= 12 * RUNS * kThreads * 8) && kShared <= 226 * 1024,
                  "room to join the rows' shares in the ring, and for the block");
    static constexpr int kBlocks = bwd_resident(kThreads, RUNS);                // on an SM
    static __device__ __forceinline__ uint8_t* narrow(uint8_t* ring, int stage, int run) {
        return ring + stage * kStage + (run * kThreads + int(threadIdx.x)) * 8;
    }
    // of the group: word w of its thread l at w kGroup + l (16 bytes each), or its words in order (4 each)
    static __device__ __forceinline__ uint8_t* wide(uint8_t* ring, int stage, int run) {
        return ring + stage * kStage + kNarrow * kThreads * 8 + (run * kGroups + int(threadIdx.x) / kGroup) * kGroupBytes;
    }
    static __device__ __forceinline__ int lane() { return int(threadIdx.x) % kGroup; }
};

// One run of a matrix of T on its way into the ring.  p: where this thread's run starts; left: how many of its values
// exist, not above zero where none does (whole runs are sent where they exist alone).  Where a 16-bit row starts in the
// middle of a word, the value before it is read with it.
template <typename R, typename T>
__device__ __forceinline__ void send(uint8_t* ring, int stage, int run, const T* p, int left) {
    uint8_t* to = R::wide(ring, stage, run);
    const int l = R::lane();
    if constexpr (R::kWhole) {
#pragma unroll
        for (int i = 0; i < R::kWords; ++i) copy_async<16>(to + (i * R::kGroup + l) * 16, p + i * (16 / sizeof(T)));
    } else {
        left += 8 * l;  // of the group
        if (left <= 0) return;
        p -= 8 * l;
        const uint8_t* q = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
        const int off = int(reinterpret_cast<const uint8_t*>(p) - q);
        constexpr int kStep = R::kGroup * 4, kAll = R::kWords * kStep;
        if (left > 8 * R::kGroup) {  // every word is the row's
#pragma unroll
            for (int i = 0; i < R::kWords; ++i) copy_async<4>(to + l * 4 + i * kStep, q + l * 4 + i * kStep);
            if (off && l == 0) copy_async<4>(to + kAll, q + kAll);
        } else {
            const int end = off + left * int(sizeof(T));
            const auto word = [&](int at) {
                const int bytes = min(max(end - at, 0), 4);
                copy_async<4>(to + at, bytes > 0 ? q + at : q, bytes);
            };
#pragma unroll
            for (int i = 0; i < R::kWords; ++i) word(l * 4 + i * kStep);
            if (sizeof(T) == 2 && l == 0) word(kAll);
        }
    }
}
// The same run out of it, zero where it is not `live`; p as it was sent from, for where in a word it starts.
template <typename R, typename T>
__device__ __forceinline__ void receive(uint8_t* ring, int stage, int run, const T* p, bool live, Run8<T>& v) {
    const uint8_t* from = R::wide(ring, stage, run);
    const int l = R::lane();
    constexpr int kQuads = int(sizeof(T)) / 2;
    uint4 w[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
        w[i] = live ? *reinterpret_cast<const uint4*>(from + (R::kWhole ? i * R::kGroup + l : l * kQuads + i) * 16)
                    : make_uint4(0u, 0u, 0u, 0u);
    if constexpr (!R::kWhole && sizeof(T) == 2) {
        const uint32_t last = live ? *reinterpret_cast<const uint32_t*>(from + (l + 1) * 16) : 0u;
        const uint32_t shift = reinterpret_cast<uintptr_t>(p) & 2 ? 16 : 0;
        w[0] = make_uint4(__funnelshift_r(w[0].x, w[0].y, shift), __funnelshift_r(w[0].y, w[0].z, shift),
                          __funnelshift_r(w[0].z, w[0].w, shift), __funnelshift_r(w[0].w, last, shift));
    }
    memcpy(&v, w, sizeof(w));
}

// A run of an operand: as it is stored, or its checkpoint's bytes and scale.
template <typename T, bool KEPT>
struct Held {
    Run8<T> v;
    __device__ __forceinline__ float2 pair(int p, float) const { return v.pair(p); }
};
template <typename T>
struct Held<T, true> {
    Bytes8 v;
    __device__ __forceinline__ float2 pair(int p, float scale) const { return f2_mul(v.pair(p), f2(scale)); }
};

// What a row has one number of, or one for each 128 columns.
template <int RUNS>
struct RowNumbers {
    float rstd_r, rstd_s, z, scales[3][RUNS];
};

enum Vector { kPost, kPre, kAlpha };

// ---- a cluster's CTAs
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// v to where p lies in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void store_there(float* p, int rank, float v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// A block takes every gridDim-th group of rows; a thread keeps the same columns throughout, so its shares of the
// vectors' gradients stay in its registers and leave once per block, to be added up in a fixed order.
//
// With 16 columns a thread those shares and what the row's two passes share take some 230 registers, so there are eight
// warps on an SM; the ring keeps memory busy all the same, and the vectors wait in shared memory, since eight warps do not
// hide loads from L1 (160,000 x 512 from checkpoints 190 against 256 us).  Measured there: three blocks an SM with spills
// 372; eight columns a thread on two warps, without the ring, 385; five rows in flight instead of two the same.  190 us is
// 5.7 TB/s, 83% of the copy's rate, and half of the instructions' rate; as stored 200 us (6.6 TB/s), float32 382 us (6.9
// TB/s), 10,007 x 1000 float16 35 us.  The vectors' gradients are 5 to 6 us of that: the partial sums' way out and the
// launch that adds them up (without them 29.5 and 183 us; 37 x 1001 float32 in a graph 5.3 of 7.4).
//
// CL: a row is a cluster's of that many CTAs, 4096 columns each; they tell each other their sums through distributed
// shared memory, one cluster barrier a row: 10,000 x 8192 bf16 from checkpoints 306 us (3.5 TB/s); one CTA that read such
// a row twice and kept its shares in shared memory took 506.
template <typename T, bool KEPT, Move MOVE, int TPR, int RUNS, int CL>
__global__ void __launch_bounds__(kBlockThreads<TPR>, (Ring<T, KEPT, MOVE, TPR, RUNS>::kBlocks))
    k_sandwich_bwd(const __grid_constant__ SandwichBwdArgs a) {
    RS_PDL_ENTER();
    using R = Ring<T, KEPT, MOVE, TPR, RUNS>;
    constexpr bool VEC = MOVE != kAny, FULL = MOVE == kFull;
    constexpr int kThreads = R::kThreads, kRows = kThreads / TPR, kStages = R::kStages;
    __shared__ float smem[2][kThreads / 32 * 3];
    __shared__ float cross[2][CL][3];
    extern __shared__ __align__(16) uint8_t ring[];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int rank = CL > 1 ? int(blockIdx.x) % CL : 0, c0 = rank * (TPR * RUNS * 8);
    const unsigned cluster = blockIdx.x / CL, clusters = gridDim.x / CL;
    const auto column = [&](int i) { return c0 + (i * TPR + t) * 8; };
    const bool element = a.gate == kElementGate;
    // The vectors, where their loads do not wait: halves of runs apart, so that neighbours hit different banks.
    float4* vectors = reinterpret_cast<float4*>(ring + R::kBytes);
    const auto vector = [&](int k, int i, float2 (&w)[4]) {
        const float4 lo = vectors[(k * 2 * RUNS + i) * TPR + t], hi = vectors[(k * 2 * RUNS + RUNS + i) * TPR + t];
        w[0] = make_float2(lo.x, lo.y), w[1] = make_float2(lo.z, lo.w);
        w[2] = make_float2(hi.x, hi.y), w[3] = make_float2(hi.z, hi.w);
    };
    float2 acc[3][RUNS][4];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < RUNS; ++i)
#pragma unroll
            for (int p = 0; p < 4; ++p) acc[k][i][p] = f2(0.f);
    // Of a run: how many of its values exist.  Widths are given to threads so that only the last run may lack some, but in a
    // cluster any.
    const auto left_of = [&](int i) { return MOVE == kAny ? a.cols - column(i) : column(i) < a.cols ? 8 : 0; };
    const auto rest = [&](int i) { return FULL || (CL == 1 && i + 1 < RUNS) ? 8 : left_of(i); };
    const auto numbers = [&](long long row) {
        RowNumbers<RUNS> n{};
        if (row >= a.rows) return n;
        n.rstd_r = a.rstd_r[row];
        n.rstd_s = a.rstd_s[row];
        if (a.gate == kRowGate) n.z = to_f(static_cast<const T*>(a.z.p)[row * a.z.stride]);
        if constexpr (KEPT) {
#pragma unroll
            for (int i = 0; i < RUNS; ++i)
                if (rest(i) > 0) {
                    const size_t at = size_t(column(i) / kBlock) * a.rows + row;
                    n.scales[0][i] = a.x.scales[at];
                    n.scales[1][i] = a.r.scales[at];
                    if (element) n.scales[2][i] = a.z.scales[at];
                }
        }
        return n;
    };
    const auto run_of = [&](const void* p, size_t stride, long long row, int i) {
        return static_cast<const T*>(p) + row * stride + column(i);
    };
    const auto operand = [&](const Stored& s, long long row, int stage, int k, int i) {
        if constexpr (KEPT) {
            if (rest(i) > 0)
                copy_async<8>(R::narrow(ring, stage, k * RUNS + i),
                              static_cast<const uint8_t*>(s.p) + row * s.stride + column(i), min(rest(i), 8));
        } else {
            send<R>(ring, stage, (2 + k) * RUNS + i, run_of(s.p, s.stride, row, i), left_of(i));
        }
    };
    const auto fetch = [&](long long row, int stage) {
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                if (R::kWhole && rest(i) <= 0) continue;
                operand(a.x, row, stage, 0, i);
                operand(a.r, row, stage, 1, i);
                if (element) operand(a.z, row, stage, 2, i);
                send<R>(ring, stage, i, run_of(a.dy, a.dys, row, i), left_of(i));
                if (a.ds) send<R>(ring, stage, RUNS + i, run_of(a.ds, a.dss, row, i), left_of(i));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const long long step = (long long)clusters * kRows;
    const long long first = (long long)cluster * kRows + sub;
    RowNumbers<RUNS> now = numbers(first);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + s * step, s);
    if (sub == 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                const float* v = k == kPost ? a.wpost : k == kPre ? a.wpre : a.alpha;
                float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
                if (v) load8<float, VEC>(v + column(i), a.cols - column(i), w);
                vectors[(k * 2 * RUNS + i) * TPR + t] = make_float4(w[0], w[1], w[2], w[3]);
                vectors[(k * 2 * RUNS + RUNS + i) * TPR + t] = make_float4(w[4], w[5], w[6], w[7]);
            }
    }
    __syncthreads();
    if constexpr (CL > 1) cluster_sync();  // the others' memory is there
    int stage = 0, turn = 0;
    for (long long base = (long long)cluster * kRows; base < a.rows; base += step) {
        const long long row = base + sub;
        const bool in = row < a.rows;
        const RowNumbers<RUNS> next = numbers(row + step);
        if constexpr (!R::kWhole) __syncwarp();   // the row before has been read by all that share its words
        fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        if constexpr (!R::kWhole) __syncwarp();   // and this one's are there
        float row_e = 0.f, row_g = 1.f;
        if (a.gate == kRowGate) {
            row_e = gate_e(now.z);
            row_g = gate_of(row_e);
        }
        Held<T, KEPT> xv[RUNS];
        float2 sh[RUNS][4], ds[RUNS][4], g[RUNS][4], rest_g[RUNS][4], rh[RUNS][4];  // rest_g: 1 - g
        float2 s0 = f2(0.f), s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const bool live = in && (FULL || rest(i) > 0);
            Held<T, KEPT> rv, zv;
            Run8<T> dy, up;
            const auto take = [&](const Stored& s, int k, Held<T, KEPT>& h) {
                if constexpr (KEPT)
                    h.v.w = live ? *reinterpret_cast<const uint2*>(R::narrow(ring, stage, k * RUNS + i)) : make_uint2(0u, 0u);
                else
                    receive<R>(ring, stage, (2 + k) * RUNS + i, run_of(s.p, s.stride, row, i), live, h.v);
            };
            take(a.x, 0, xv[i]);
            take(a.r, 1, rv);
            if (element) take(a.z, 2, zv);
            receive<R>(ring, stage, i, run_of(a.dy, a.dys, row, i), live, dy);
            if (a.ds) receive<R>(ring, stage, RUNS + i, run_of(a.ds, a.dss, row, i), live, up);
            if (element) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float2 e = gate_e(zv.pair(p, now.scales[2][i]));
                    g[i][p] = gate_of(e);
                    rest_g[i][p] = f2_mul(e, g[i][p]);
                }
            } else {
#pragma unroll
                for (int p = 0; p < 4; ++p) g[i][p] = f2(row_g), rest_g[i][p] = f2(row_e * row_g);
            }
            float2 w[4];
            vector(kPost, i, w);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                rh[i][p] = f2_mul(rv.pair(p, now.scales[1][i]), f2(now.rstd_r));
                w[p] = f2_mul(g[i][p], f2_mul(rh[i][p], w[p]));                      // p
            }
            float2 al[4];
            vector(kAlpha, i, al);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                sh[i][p] = f2_mul(f2_fma(al[p], xv[i].pair(p, now.scales[0][i]), w[p]), f2(now.rstd_s));
                s2 = f2_fma(sh[i][p], w[p], s2);
            }
            vector(kPre, i, al);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float2 d = dy.pair(p), t = f2_mul(d, al[p]);
                acc[0][i][p] = f2_fma(d, sh[i][p], acc[0][i][p]);
                s0 = f2_fma(t, sh[i][p], s0);
                ds[i][p] = f2_fma(f2(now.rstd_s), t, a.ds ? up.pair(p) : f2(0.f));
                s1 = f2_fma(ds[i][p], w[p], s1);
            }
        }
        float sums[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
        row_sums<TPR>(sums, smem[turn ^= 1]);
        if constexpr (CL > 1) {
            if (t < CL)
#pragma unroll
                for (int k = 0; k < 3; ++k) store_there(&cross[turn][rank][k], t, sums[k]);
            __syncwarp();
            cluster_sync();  // (the row after the next uses this memory again: all have read it by the next one's barrier)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                sums[k] = cross[turn][0][k];
#pragma unroll
                for (int i = 1; i < CL; ++i) sums[k] += cross[turn][i][k];
            }
        }
        const float c1 = now.rstd_s * (sums[0] * a.inv_cols);
        const float dot = fmaf(-c1, sums[2], sums[1]);           // sum of ds p
        const float c2 = dot * a.inv_cols;
        if (a.gate == kRowGate && a.dz && in && t == 0 && rank == 0)
            static_cast<T*>(a.dz)[row * a.dzs] = from_f<T>(dot * (row_e * row_g));
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int left = in ? rest(i) : 0;
            float2 w[4], o[4], dn[4];
            vector(kAlpha, i, w);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                ds[i][p] = f2_fma(f2(-c1), sh[i][p], ds[i][p]);
                acc[2][i][p] = f2_fma(ds[i][p], xv[i].pair(p, now.scales[0][i]), acc[2][i][p]);
                dn[p] = f2_mul(ds[i][p], g[i][p]);
                acc[1][i][p] = f2_fma(dn[p], rh[i][p], acc[1][i][p]);
                o[p] = f2_mul(ds[i][p], w[p]);
            }
            if (left > 0) store_pairs<T, VEC>(static_cast<T*>(a.dx) + row * a.dxs + column(i), left, o);
            vector(kPost, i, w);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                dn[p] = f2_mul(dn[p], w[p]);
                o[p] = f2_mul(f2(now.rstd_r), f2_fma(f2(-c2), rh[i][p], dn[p]));
                dn[p] = f2_mul(f2_mul(dn[p], rh[i][p]), rest_g[i][p]);
            }
            if (left > 0) {
                store_pairs<T, VEC>(static_cast<T*>(a.dr) + row * a.drs + column(i), left, o);
                if (element && a.dz) store_pairs<T, VEC>(static_cast<T*>(a.dz) + row * a.dzs + column(i), left, dn);
            }
        }
        now = next;
        if (++stage == kStages) stage = 0;
    }
    if (!a.part) return;
    float* part = a.part + size_t(cluster) * 3 * a.cols;
    const auto leave = [&](int k, int i, int p, float2 v) {
        const int c = column(i) + 2 * p;
        if (c < a.cols) part[size_t(k) * a.cols + c] = v.x;
        if (c + 1 < a.cols) part[size_t(k) * a.cols + c + 1] = v.y;
    };
    if constexpr (kRows == 1) {
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < RUNS; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) leave(k, i, p, acc[k][i][p]);
    } else {  // the rows' threads join their shares, each some of them
        float2* comb = reinterpret_cast<float2*>(ring);  // no copy is on its way to it: no row is left
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < RUNS; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) comb[((k * RUNS + i) * 4 + p) * kThreads + threadIdx.x] = acc[k][i][p];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 12 * RUNS; ++n) {
            if (n % kRows != sub) continue;
            float2 v = comb[n * kThreads + t];
            for (int o = 1; o < kRows; ++o) {
                const float2 w = comb[n * kThreads + o * TPR + t];
                v = make_float2(v.x + w.x, v.y + w.y);
            }
            leave(n / (4 * RUNS), n / 4 % RUNS, n % 4, v);
        }
    }
}

struct Vectors { float* out[3]; };

// The vectors' gradients from the blocks' sums [n][3][cols] in a fixed order: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(1024) k_sandwich_sums(const float* __restrict__ part, int n, int cols, Vectors v) {
    RS_PDL_ENTER();
    float* out = v.out[blockIdx.y];
    if (!out) return;
    __shared__ float sm[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float s = 0.f;
    if (c < cols)
#pragma unroll 8
        for (int i = g; i < n; i += 32) s += part[(size_t(i) * 3 + blockIdx.y) * cols + c];
    sm[g][threadIdx.x & 31] = s;
    __syncthreads();
    s = group_sum<32>(sm[threadIdx.x & 31][g]);
    const int oc = blockIdx.x * 32 + g;
    if ((threadIdx.x & 31) == 0 && oc < cols) out[oc] = s;
}

// How many clusters the GPU holds at once (a grid of more would run in two turns).  Asked in every call: the answer is the
// current device's, and a question that failed once may not decide later calls.
template <typename K>
cudaError_t clusters_at_once(K kernel, int cluster, int threads, int smem, int& n) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = cluster;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
}

template <typename T, bool KEPT, Move MOVE, int TPR, int RUNS, int CL>
cudaError_t bwd(const SandwichBwdArgs& a, unsigned& parts, cudaStream_t s) {
    using R = Ring<T, KEPT, MOVE, TPR, RUNS>;
    const auto kernel = k_sandwich_bwd<T, KEPT, MOVE, TPR, RUNS, CL>;
    if (R::kShared > 47 * 1024) {  // with what is static, more than needs no leave
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kShared);
        if (e != cudaSuccess) return e;
    }
    int most = kSms * R::kBlocks;
    if constexpr (CL > 1) {
        int at_once;
        const cudaError_t e = clusters_at_once(kernel, CL, R::kThreads, R::kShared, at_once);
        if (e != cudaSuccess) return e;
        if (at_once < 1) return cudaErrorInvalidConfiguration;
        most = std::min(at_once, kSms / CL);
    }
    parts = unsigned(std::min(ceil_div(a.rows, R::kThreads / TPR), most));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = parts * CL;
    cfg.blockDim = R::kThreads;
    cfg.dynamicSmemBytes = R::kShared;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, bool KEPT, Move MOVE>
cudaError_t bwd_width(const SandwichBwdArgs& a, unsigned& parts, cudaStream_t s) {
    switch (bwd_ctas(a.cols)) {
        case 2: return bwd<T, KEPT, MOVE, 256, 2, 2>(a, parts, s);
        case 4: return bwd<T, KEPT, MOVE, 256, 2, 4>(a, parts, s);
    }
    const Shape p = bwd_shape(a.cols, sizeof(T) == 4);
    if constexpr (sizeof(T) == 2) {
        switch (p.threads) {
            case 96: return bwd<T, KEPT, MOVE, 96, 1, 1>(a, parts, s);
            case 192: return bwd<T, KEPT, MOVE, 192, 1, 1>(a, parts, s);
            case 384: return bwd<T, KEPT, MOVE, 384, 1, 1>(a, parts, s);
        }
    }
    switch (p.threads) {
        case 16: return p.runs == 1 ? bwd<T, KEPT, MOVE, 16, 1, 1>(a, parts, s) : bwd<T, KEPT, MOVE, 16, 2, 1>(a, parts, s);
        case 32: return bwd<T, KEPT, MOVE, 32, 2, 1>(a, parts, s);
        case 64: return bwd<T, KEPT, MOVE, 64, 2, 1>(a, parts, s);
        case 128: return bwd<T, KEPT, MOVE, 128, 2, 1>(a, parts, s);
    }
    return bwd<T, KEPT, MOVE, 256, 2, 1>(a, parts, s);
}

}  // namespace
}  // namespace rs

extern "C" {

size_t rs_sandwich_norm_bwd_workspace_size(int32_t rows, int32_t cols) {
    if (rows < 0 || cols < 1 || cols > RS_NORM_MAX_COLS) return 0;
    const int blocks = std::max({1, rs::bwd_blocks(rows, cols, false), rs::bwd_blocks(rows, cols, true)});  // whatever the type
    return size_t(blocks) * 3 * cols * sizeof(float);
}

int rs_sandwich_norm_bwd(const rs_sandwich* block, const rs_sandwich_grads* grads, void* d_workspace,
                         size_t workspace_bytes, void* stream) {
    using namespace rs;
    if (!block || !grads) return RS_ERR_INVALID_ARG;
    bool kept, vec;
    if (!operands_ok(block, kept, vec)) return RS_ERR_INVALID_ARG;
    const int32_t rows = block->rows, cols = block->cols, dtype = block->dtype;
    const size_t z = dtype_size(dtype);
    float* const vectors[3] = {grads->d_dL_dpre_weight, grads->d_dL_dpost_weight, grads->d_dL_dresidual_scale};
    bool any = false;
    for (float* v : vectors) {
        if (v && !ptr_ok(v, 4)) return RS_ERR_INVALID_ARG;
        any = any || v;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        for (float* v : vectors)
            if (v && cudaMemsetAsync(v, 0, size_t(cols) * 4, s) != cudaSuccess) return RS_ERR_CUDA;
        return RS_OK;
    }
    if (!ptr_ok(grads->d_rstd_r, 4) || !ptr_ok(grads->d_rstd_s, 4)) return RS_ERR_INVALID_ARG;
    struct Out { void* p; size_t stride; };
    const Out in[2] = {{const_cast<void*>(grads->d_dL_dy), grads->dy_stride},
                       {const_cast<void*>(grads->d_dL_dsum), grads->dsum_stride}};
    const Out out[3] = {{grads->d_dL_dx, grads->dx_stride}, {grads->d_dL_dr, grads->dr_stride},
                        {grads->d_dL_dgate, grads->dgate_stride}};
    if (!matrix_ok(in[0].p, in[0].stride, cols, dtype) || (in[1].p && !matrix_ok(in[1].p, in[1].stride, cols, dtype)))
        return RS_ERR_INVALID_ARG;
    if (out[2].p && !block->gate_cols) return RS_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        if (i == 2 && !out[2].p) break;
        const int32_t width = i == 2 ? block->gate_cols : cols;
        if (!matrix_ok(out[i].p, out[i].stride, width, dtype)) return RS_ERR_INVALID_ARG;
        for (const Out& o : in)
            if (o.p == out[i].p && (o.stride != out[i].stride || width != cols)) return RS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[j].p == out[i].p) return RS_ERR_INVALID_ARG;
        if (width == cols) vec = vec && rows16(out[i].p, out[i].stride, z);
    }
    for (const Out& o : in)
        if (o.p) vec = vec && rows16(o.p, o.stride, z);
    if (any) {
        if (!ptr_ok(d_workspace, 16)) return RS_ERR_INVALID_ARG;
        if (workspace_bytes < rs_sandwich_norm_bwd_workspace_size(rows, cols)) return RS_ERR_WORKSPACE;
    }
    const SandwichBwdArgs a{args_of(block), grads->d_rstd_r, grads->d_rstd_s, in[0].p, in[0].stride, in[1].p,
                            in[1].stride, out[0].p, out[0].stride, out[1].p, out[1].stride, out[2].p, out[2].stride,
                            any ? static_cast<float*>(d_workspace) : nullptr};
    unsigned parts = 0;
    cudaError_t e = with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        // nothing asked, as in the forward, pays from checkpoints alone (160,000 x 512: 190 us, 196 asking; as stored 214
        // and 206)
        if (kept) {
            if (!vec) return bwd_width<T, true, kAny>(a, parts, s);
            const Shape p = bwd_shape(cols, dtype == RS_F32);
            return cols == 8 * p.threads * p.runs * bwd_ctas(cols) ? bwd_width<T, true, kFull>(a, parts, s)
                                                                   : bwd_width<T, true, kRuns>(a, parts, s);
        }
        return vec ? bwd_width<T, false, kRuns>(a, parts, s) : bwd_width<T, false, kAny>(a, parts, s);
    });
    if (e == cudaSuccess && any)
        e = pdl_launch(k_sandwich_sums, dim3(ceil_div(cols, 32), 3), 1024, 0, s, static_cast<const float*>(a.part),
                       int(parts), cols, Vectors{{vectors[0], vectors[1], vectors[2]}});
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
