// The norms before and after a residual block, with the block's gate and the residual scale, and their backward.
//
// Per row:  rh = r rstd_r,  s = alpha x + g rh wpost,  g = 1 / (1 + exp(-z)),  y = s rstd_s wpre, with rstd_r and rstd_s
// the reciprocal root mean squares of r and s; y leaves in 8 bits, and so do x, r and z where the backward is to read
// them from there.
//
// Backward, with t = dy wpre, sh = s rstd_s, p = g rh wpost:
//   ds = rstd_s (t - sh mean(t sh)) + dsum,   dx = alpha ds,   dr = rstd_r (ds g wpost - rh mean(ds p)),
//   dz = ds p (1 - g),   dalpha = sum ds x,   dwpost = sum ds g rh,   dwpre = sum dy sh.
// mean(ds p) seems to need ds, and that mean(t sh); but it is linear in ds:
//   sum ds p = sum (rstd_s t + dsum) p - rstd_s mean(t sh) sum sh p,
// so that one pass over the row gives all three sums.
#pragma once

#include "sandwich_plan.h"
#include "wide.cuh"

namespace rs {
namespace {

struct Stored { const void* p; size_t stride; const float* scales; };  // scales: e4m3 with a scale per 128 columns
struct Form { uint8_t* q; size_t stride; float* scales; };

struct SandwichArgs {
    int rows, cols, gate;                 // gate: 0 none, 1 one a row, 2 one an element
    Stored x, r, z;
    const float* alpha;
    const float* wpost;
    const float* wpre;
    float inv_cols;
    bool wide;                            // the vectors start on 16-byte boundaries
};

struct SandwichFwdArgs : SandwichArgs {
    float eps;
    void* sum; size_t sums;
    void* y; size_t ys;
    Form q, kx, kr, kz;
    float* rstd_r;
    float* rstd_s;
};

struct SandwichBwdArgs : SandwichArgs {
    const float* rstd_r;
    const float* rstd_s;
    const void* dy; size_t dys;
    const void* ds; size_t dss;
    void* dx; size_t dxs;
    void* dr; size_t drs;
    void* dz; size_t dzs;
    float* part;                          // [blocks][3][cols]: a block's sums for wpre, wpost, alpha
};

constexpr int kNoGate = 0, kRowGate = 1, kElementGate = 2;

// exp(-z) of a gate, held below exp(80) so that g = 1 / (1 + e) and 1 - g = e g are numbers whatever z is (NaN stays):
// gates below 1.8e-35 count as that.  (The forward keeps z within 80 of zero, too, so that an infinity or a type's lowest
// value is no block's largest magnitude: that would leave the block's other gates no bits, or NaN.)  2^x and 1 / x to
// within two of their last bits, without the steps that would carry results below 2^-126: e near zero adds nothing to 1,
// and 1 + e is at most 2^116.
constexpr float kGateEnd = 80.f;
__device__ __forceinline__ float gate_e(float z) {
    constexpr float kLog2E = 1.44269504f;
    float e;
    asm("{\n .reg .f32 x;\n min.NaN.f32 x, %1, %2;\n ex2.approx.ftz.f32 %0, x;\n}\n"
        : "=f"(e) : "f"(z * -kLog2E), "f"(kGateEnd * kLog2E));
    return e;
}
__device__ __forceinline__ float gate_of(float e) {
    float g;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(1.f + e));
    return g;
}
__device__ __forceinline__ float2 gate_e(float2 z) { return make_float2(gate_e(z.x), gate_e(z.y)); }
__device__ __forceinline__ float2 gate_of(float2 e) { return make_float2(gate_of(e.x), gate_of(e.y)); }

// A barrier of the TPR threads of a row, in a block of THREADS.  Two rows of 64 do not wait for each other.  (The
// barriers' numbers stand in the code: with a number from a register a block holds all sixteen, and few blocks fit an
// SM: 80,000 x 1000 bf16 forward 286 us, with one barrier for both rows 203.)
template <int TPR, int THREADS>
__device__ __forceinline__ void row_barrier() {
    static_assert(TPR == THREADS || (TPR == 64 && THREADS == 128), "whole warps");
    if (TPR == THREADS) __syncthreads();
    else if (threadIdx.x < TPR) asm volatile("bar.sync 1, 64;" ::: "memory");
    else asm volatile("bar.sync 2, 64;" ::: "memory");
}

// Sums over the TPR threads of a row.  All of them call it (TPR > 32 uses a barrier, and the call after the next may use
// the same memory again).
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* smem) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = group_sum<(TPR < 32 ? TPR : 32)>(v[k]);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) smem[(threadIdx.x >> 5) * N + k] = v[k];
        row_barrier<TPR, kBlockThreads<TPR>>();
        const float* mine = smem + threadIdx.x / TPR * kWarps * N;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) v[k] += mine[i * N + k];
        }
    }
}

// How a row is moved: value by value or word by word; in 16-byte accesses (rows on such boundaries, whole runs of eight:
// a thread has a run or has none); or in such accesses by threads that all have theirs (the width is 8 TPR RUNS).
enum Move { kAny, kRuns, kFull };

// Eight values of a vector; `wide`: it starts on a 16-byte boundary (value by value the loads of neighbours' runs take
// eight times the L1's turns, 80,000 x 1001 bf16 forward 394 against 338 us).
template <bool VEC>
__device__ __forceinline__ void load_vector(const float* p, int left, bool wide, float2 (&v)[4]) {
    float w[8];
    if (VEC || wide) load8<float, true>(p, left, w);
    else load8<float, false>(p, left, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(w[2 * i], w[2 * i + 1]);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_pairs(T* p, int left, const float2 (&v)[4]) {
    const float w[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    store8<T, VEC>(p, left, w);
}
// ---------------------------------------------------------------- host side
bool matrix_ok(const void* p, size_t stride, int32_t cols, int32_t dtype) {
    return ptr_ok(p, dtype_size(dtype)) && stride >= size_t(cols);
}
bool form_ok(const rs_fp8_matrix& f, int32_t cols) {
    if (!f.d_q && !f.d_scales) return true;
    return fp8_rows_ok(f.d_q, f.stride, cols) && ptr_ok(f.d_scales, 4);
}

bool wide_vectors(const rs_sandwich* b) {
    return ptr_ok(b->d_post_weight, 16) && ptr_ok(b->d_pre_weight, 16) &&
           (!b->d_residual_scale || ptr_ok(b->d_residual_scale, 16));
}

// The block's operands; `kept`: whether they are checkpoints, `vec`: whether runs can move in 16-byte accesses.
bool operands_ok(const rs_sandwich* b, bool& kept, bool& vec) {
    if (b->rows < 0 || b->cols < 1 || b->cols > RS_NORM_MAX_COLS || !dtype_ok(b->dtype)) return false;
    if (b->gate_cols != 0 && b->gate_cols != 1 && b->gate_cols != b->cols) return false;
    kept = b->d_x_scales != nullptr;
    vec = true;
    if (b->rows == 0) return true;
    if (!ptr_ok(b->d_post_weight, 4) || !ptr_ok(b->d_pre_weight, 4)) return false;
    if (b->d_residual_scale && !ptr_ok(b->d_residual_scale, 4)) return false;
    if (kept != (b->d_r_scales != nullptr)) return false;
    const size_t z = dtype_size(b->dtype);
    const bool element = b->gate_cols > 1;
    if (kept) {
        if (!fp8_rows_ok(b->d_x, b->x_stride, b->cols) || !fp8_rows_ok(b->d_r, b->r_stride, b->cols)) return false;
        if (!ptr_ok(b->d_x_scales, 4) || !ptr_ok(b->d_r_scales, 4)) return false;
    } else if (!matrix_ok(b->d_x, b->x_stride, b->cols, b->dtype) || !matrix_ok(b->d_r, b->r_stride, b->cols, b->dtype)) {
        return false;
    }
    if (b->gate_cols) {
        if ((b->d_gate_scales != nullptr) != (kept && element)) return false;
        if (kept && element) {
            if (!fp8_rows_ok(b->d_gate, b->gate_stride, b->cols) || !ptr_ok(b->d_gate_scales, 4)) return false;
        } else if (!matrix_ok(b->d_gate, b->gate_stride, b->gate_cols, b->dtype)) {
            return false;
        }
    }
    vec = b->cols % 8 == 0 && wide_vectors(b);
    if (!kept)
        vec = vec && rows16(b->d_x, b->x_stride, z) && rows16(b->d_r, b->r_stride, z) &&
              (!element || rows16(b->d_gate, b->gate_stride, z));
    return true;
}

SandwichArgs args_of(const rs_sandwich* b) {
    return {b->rows, b->cols, b->gate_cols == 0 ? kNoGate : b->gate_cols == 1 ? kRowGate : kElementGate,
            {b->d_x, b->x_stride, b->d_x_scales}, {b->d_r, b->r_stride, b->d_r_scales},
            {b->d_gate, b->gate_stride, b->d_gate_scales}, b->d_residual_scale, b->d_post_weight, b->d_pre_weight,
            1.0f / float(b->cols), wide_vectors(b)};
}

}  // namespace
}  // namespace rs
