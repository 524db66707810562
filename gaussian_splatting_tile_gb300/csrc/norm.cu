// Root-mean-square norm with the residual's addition and an 8-bit output, and its backward.
//
// Forward, per row: s = x + r, rstd = 1 / sqrt(mean s^2 + eps), y = s rstd w, then per 128 columns the largest |y|
// gives a scale and y becomes e4m3.  Everything is bound by memory: x, r in, s and q out, 7 bytes a value in 16 bits.
// So a row stays in registers between the two sums: TPR threads hold it as runs of eight consecutive values (16 bytes
// of a 16-bit type), and a block of 128 columns is the run of 16 neighbouring threads, whose maximum takes four
// shuffles.  The norm is taken of the sum before its rounding to 16 bits.
//
// Measured (GB300, inputs beyond L2): 250,000 x 512 bf16 with the residual 128 us (7.0 TB/s; the copy 6.7), float32
// 6.9 TB/s; 160,000 x 1000 bf16, whose rows end inside a thread's runs, 5.4 TB/s. Rows that do not start on 16-byte
// boundaries go by words: 100,000 x 777 bf16 2.6 TB/s.  One row of 4096 costs the call (9 us).
//
// Backward, per row: xh = s rstd, t = dy w, dx = rstd (t - xh mean(t xh)) + ds; dw = sum over rows of dy xh.  Bound
// by memory too: three matrices in, one out.  160,000 x 256 float32 103 us (6.3 TB/s), 160,000 x 512 bf16 5.4 TB/s.
#include "wide.cuh"

namespace rs {
namespace {

struct NormArgs {
    int rows, cols;
    const void* x; size_t xs;
    const void* r; size_t rs_;
    const float* w;
    float eps, inv_cols;
    void* sum; size_t sums;
    void* y; size_t ys;
    uint8_t* q; size_t qs;
    float* scales;
    float* rstd;
};

// Sum over the TPR threads of a row.  All threads of the block call it (TPR > 32 uses barriers).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* smem) {
    v = group_sum<(TPR < 32 ? TPR : 32)>(v);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
        const float* mine = smem + threadIdx.x / TPR * kWarps;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) v += mine[i];
    }
    return v;
}

// How a row is moved: value by value or word by word, in 16-byte accesses with a ragged end, or all of it in such
// accesses (the width is 8 TPR RUNS).
enum Move { kAny, kVec, kFull };

template <typename T, Move MOVE, int TPR, int RUNS>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_rms_norm_fwd(NormArgs a) {
    RS_PDL_ENTER();
    constexpr bool VEC = MOVE != kAny;
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    __shared__ float smem[32];
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool in = row < a.rows;
    const T* x = static_cast<const T*>(a.x) + (in ? row : 0) * a.xs;
    const T* r = a.r ? static_cast<const T*>(a.r) + (in ? row : 0) * a.rs_ : nullptr;
    float v[RUNS][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int c = (i * TPR + t) * 8, left = MOVE == kFull ? 8 : in ? a.cols - c : 0;
        load8<T, VEC>(x + c, left, v[i], c > 0);
        if (r) {
            float u[8];
            load8<T, VEC>(r + c, left, u, c > 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += u[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(ss, smem) * a.inv_cols + a.eps);
    if (in && t == 0 && a.rstd) a.rstd[row] = rstd;
    if (a.sum && in) {
        T* s = static_cast<T*>(a.sum) + row * a.sums;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int c = (i * TPR + t) * 8;
            store8<T, VEC>(s + c, MOVE == kFull ? 8 : a.cols - c, v[i]);
        }
    }
    float top[RUNS];
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int c = (i * TPR + t) * 8, left = MOVE == kFull ? 8 : in ? a.cols - c : 0;
        float w[8];
        load8<float, VEC>(a.w + c, left, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
        if (a.y && in && left > 0) store8<T, VEC>(static_cast<T*>(a.y) + row * a.ys + c, left, v[i]);
        top[i] = group_max<16>(max_abs8(v[i], 0.f));
    }
    if (!a.q) return;
    // thread i of the sixteen that share a block's columns forms run i's two quotients, and passes them on
    const int of = t & 15;
    float mine = top[0], scale, inv;
#pragma unroll
    for (int i = 1; i < RUNS; ++i) mine = of == i ? top[i] : mine;
    block_scale(mine, scale, inv);
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int c = (i * TPR + t) * 8, left = MOVE == kFull ? 8 : a.cols - c;
        const float k = __shfl_sync(0xffffffffu, inv, i, 16);
        if (of == i && in && (MOVE == kFull || c - of * 8 < a.cols))
            a.scales[size_t(c / kBlock) * a.rows + row] = scale;
        if (in && left > 0) store8_e4m3(a.q + row * a.qs + c, left, v[i], k);
    }
}

template <typename T, Move MOVE, int TPR, int RUNS>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    return pdl_launch(k_rms_norm_fwd<T, MOVE, TPR, RUNS>, ceil_div(a.rows, kRows), TPR < 128 ? 128 : TPR, 0, s, a);
}

// Widths that two or three runs for each of 16, 32, ... 512 threads fit exactly (and 128): no run asks whether it
// exists, which is a third of the instructions (bf16 with the residual: 250,000 x 512 136 us, 158 with the questions;
// 160,000 x 768 132 against 189, x 1024 171 against 197).
template <typename T, int TPR>
cudaError_t fwd_two_three(const NormArgs& a, cudaStream_t s) {
    return a.cols == TPR * 16 ? fwd<T, kFull, TPR, 2>(a, s) : fwd<T, kFull, TPR, 3>(a, s);
}

template <typename T>
cudaError_t fwd_exact(const NormArgs& a, cudaStream_t s, bool& taken) {
    const int runs = a.cols / 8, each = runs % 3 == 0 ? 3 : 2, threads = runs / each;
    taken = a.cols % 8 == 0 && threads * each == runs;
    if (taken) switch (threads) {
        case 16: return fwd_two_three<T, 16>(a, s);
        case 32: return fwd_two_three<T, 32>(a, s);
        case 64: return fwd_two_three<T, 64>(a, s);
        case 128: return fwd_two_three<T, 128>(a, s);
        case 256: return fwd_two_three<T, 256>(a, s);
        case 512: return fwd_two_three<T, 512>(a, s);
        case 8: if (each == 2) return fwd<T, kFull, 16, 1>(a, s);
    }
    taken = false;
    return cudaSuccess;
}

// Other widths: threads a row and runs a thread, measured with the residual in bf16: 250,000 x 512 on a warp 158 us,
// on two with one run each the same (without a residual 105 against 132), on half a warp 203; 160,000 x 1000 on four
// warps 208, on two 224, on one 267; 30,000 x 4096 on eight 171, on sixteen 179, on four 195.
template <typename T, Move MOVE>
cudaError_t fwd_width(const NormArgs& a, cudaStream_t s) {
    const int runs = ceil_div(a.cols, 8);
    if (runs <= 16) return fwd<T, MOVE, 16, 1>(a, s);
    if (runs <= 32) return fwd<T, MOVE, 32, 1>(a, s);
    if (runs <= 64) return fwd<T, MOVE, 32, 2>(a, s);
    if (runs <= 128) return fwd<T, MOVE, 128, 1>(a, s);
    if (runs <= 256) return fwd<T, MOVE, 128, 2>(a, s);
    if (runs <= 512) return fwd<T, MOVE, 256, 2>(a, s);
    if (runs <= 1024) return fwd<T, MOVE, 512, 2>(a, s);
    return fwd<T, MOVE, 512, 4>(a, s);
}

// ---------------------------------------------------------------- backward
struct NormBwdArgs {
    int rows, cols;
    const void* s; size_t ss;
    const float* w;
    const float* rstd;
    const void* dy; size_t dys;
    const void* ds; size_t dss;
    void* dx; size_t dxs;
    float* part;                    // [blocks][cols]: each block's sum of dy xh, nullptr: not wanted
    float inv_cols;
};

// A block takes every gridDim-th group of rows; a thread keeps the same columns throughout, so its share of
// dL/dweight stays in registers and leaves once per block, to be added up in a fixed order.  What keeps the memory
// busy is the number of rows in flight on an SM; asking for the next row's values ahead took registers, and blocks,
// and was slower (160,000 x 512 bf16 128 against 121 us), as were four runs a thread (100,000 x 1000 bf16 541 us).
template <typename T, bool VEC, int TPR, int RUNS>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_rms_norm_bwd(NormBwdArgs a) {
    RS_PDL_ENTER();
    constexpr int kThreads = TPR < 128 ? 128 : TPR;
    constexpr int kRows = kThreads / TPR;
    __shared__ float smem[32];
    __shared__ float comb[kRows > 1 ? kThreads * 8 : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float dw[RUNS][8];
#pragma unroll
    for (int i = 0; i < RUNS; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    for (long long base = (long long)blockIdx.x * kRows; base < a.rows; base += (long long)gridDim.x * kRows) {
        const long long row = base + sub;
        const bool in = row < a.rows;
        const long long rr = in ? row : 0;
        const float rstd = in ? a.rstd[rr] : 0.f;
        const T* s = static_cast<const T*>(a.s) + rr * a.ss;
        const T* dy = static_cast<const T*>(a.dy) + rr * a.dys;
        const T* ds = a.ds ? static_cast<const T*>(a.ds) + rr * a.dss : nullptr;
        // everything that the row needs is asked for at once; s, dy and ds wait as they are stored
        Run8<T> sv[RUNS], gv[RUNS], dv[RUNS];
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int c = (i * TPR + t) * 8, left = in ? a.cols - c : 0;
            sv[i].template load<VEC>(s + c, left, c > 0);
            gv[i].template load<VEC>(dy + c, left, c > 0);
            if (ds) dv[i].template load<VEC>(ds + c, left, c > 0);
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int c = (i * TPR + t) * 8;
            float w[8];
            load8<float, VEC>(a.w + c, a.cols - c, w);  // from L1: registers for it would cost a block of the SM
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float2 x = sv[i].pair(p), g = gv[i].pair(p);
                const float x0 = x.x * rstd, x1 = x.y * rstd;
                dw[i][2 * p] = fmaf(g.x, x0, dw[i][2 * p]);
                dw[i][2 * p + 1] = fmaf(g.y, x1, dw[i][2 * p + 1]);
                dot = fmaf(g.x * w[2 * p], x0, dot);
                dot = fmaf(g.y * w[2 * p + 1], x1, dot);
            }
        }
        const float c1 = row_sum<TPR>(dot, smem) * a.inv_cols;
        if (in) {
            T* dx = static_cast<T*>(a.dx) + row * a.dxs;
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                const int c = (i * TPR + t) * 8, left = a.cols - c;
                float o[8], w[8];
                load8<float, VEC>(a.w + c, left, w);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float2 x = sv[i].pair(p), g = gv[i].pair(p);
                    const float2 d = ds ? dv[i].pair(p) : make_float2(0.f, 0.f);
                    o[2 * p] = fmaf(rstd, g.x * w[2 * p] - x.x * rstd * c1, d.x);
                    o[2 * p + 1] = fmaf(rstd, g.y * w[2 * p + 1] - x.y * rstd * c1, d.y);
                }
                store8<T, VEC>(dx + c, left, o);
            }
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int c = (i * TPR + t) * 8;
        if constexpr (kRows > 1) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) comb[threadIdx.x * 8 + j] = dw[i][j];
            __syncthreads();
            if (sub == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    for (int k = 1; k < kRows; ++k) dw[i][j] += comb[(k * TPR + t) * 8 + j];
        }
        if (sub == 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < a.cols) a.part[size_t(blockIdx.x) * a.cols + c + j] = dw[i][j];
    }
}

// Column sums of part [n][cols] in a fixed order: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(1024) k_column_sums(const float* __restrict__ part, int n, int cols,
                                                      float* __restrict__ out) {
    RS_PDL_ENTER();
    __shared__ float sm[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float v = 0.f;
    if (c < cols)
#pragma unroll 8
        for (int i = g; i < n; i += 32) v += part[size_t(i) * cols + c];
    sm[g][threadIdx.x & 31] = v;
    __syncthreads();
    v = group_sum<32>(sm[threadIdx.x & 31][g]);
    const int oc = blockIdx.x * 32 + g;
    if ((threadIdx.x & 31) == 0 && oc < cols) out[oc] = v;
}

// Threads a row and blocks an SM for a width: as many blocks as fit at once, with the rows in flight that their
// registers leave room for (a thread's share of dL/dweight among them).  One run a thread up to 512 columns and from
// 1025 to 2048 (60,000 x 2048 bf16 194 us, with two 204), two otherwise (100,000 x 1000 bf16 156 us, with one 184;
// 30,000 x 4096 206 against 236).
int bwd_threads(int cols) {
    const int runs = ceil_div(cols, 8);
    return runs <= 16 ? 16 : runs <= 32 ? 32 : runs <= 128 ? 64 : runs <= 512 ? 256 : 512;
}
int bwd_blocks(int rows, int cols) {
    const int t = bwd_threads(cols), rows_a_block = t < 128 ? 128 / t : 1;
    const int per = cols <= 512 ? 8 : t == 64 ? 5 : cols <= 2048 ? 4 : t == 256 ? 2 : 1;
    return std::max(1, std::min(ceil_div(rows, rows_a_block), kSms * per));
}

template <typename T, bool VEC, int TPR, int RUNS>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t s) {
    return pdl_launch(k_rms_norm_bwd<T, VEC, TPR, RUNS>, bwd_blocks(a.rows, a.cols), TPR < 128 ? 128 : TPR, 0, s, a);
}

template <typename T, bool VEC>
cudaError_t bwd_width(const NormBwdArgs& a, cudaStream_t s) {
    switch (bwd_threads(a.cols)) {
        case 16: return bwd<T, VEC, 16, 1>(a, s);
        case 32: return bwd<T, VEC, 32, 1>(a, s);
        case 64: return a.cols <= 512 ? bwd<T, VEC, 64, 1>(a, s) : bwd<T, VEC, 64, 2>(a, s);
        case 256: return a.cols <= 2048 ? bwd<T, VEC, 256, 1>(a, s) : bwd<T, VEC, 256, 2>(a, s);
    }
    return a.cols <= 8192 ? bwd<T, VEC, 512, 2>(a, s) : bwd<T, VEC, 512, 4>(a, s);
}

bool matrix_ok(const void* p, size_t stride, int32_t cols, int32_t dtype) {
    return ptr_ok(p, dtype_size(dtype)) && stride >= size_t(cols);
}

}  // namespace
}  // namespace rs

extern "C" {

int rs_rms_norm_fwd(int32_t rows, int32_t cols, int32_t dtype, const void* d_x, size_t x_stride,
                    const void* d_residual, size_t residual_stride, const float* d_weight, float eps, void* d_sum,
                    size_t sum_stride, void* d_y, size_t y_stride, uint8_t* d_q, size_t q_stride, float* d_scales,
                    float* d_rstd, void* stream) {
    using namespace rs;
    if (rows < 0 || cols < 1 || cols > RS_NORM_MAX_COLS || !dtype_ok(dtype) || !(eps >= 0.f) || !isfinite(eps))
        return RS_ERR_INVALID_ARG;
    if (rows == 0) return RS_OK;
    const size_t z = dtype_size(dtype);
    if (!matrix_ok(d_x, x_stride, cols, dtype) || !ptr_ok(d_weight, 4)) return RS_ERR_INVALID_ARG;
    if (d_residual && !matrix_ok(d_residual, residual_stride, cols, dtype)) return RS_ERR_INVALID_ARG;
    if (d_sum && !matrix_ok(d_sum, sum_stride, cols, dtype)) return RS_ERR_INVALID_ARG;
    if (d_sum && ((d_sum == d_x && sum_stride != x_stride) || (d_sum == d_residual && sum_stride != residual_stride)))
        return RS_ERR_INVALID_ARG;
    if (d_y && !matrix_ok(d_y, y_stride, cols, dtype)) return RS_ERR_INVALID_ARG;
    if ((d_q == nullptr) != (d_scales == nullptr) || (!d_q && !d_y)) return RS_ERR_INVALID_ARG;
    if (d_q && (!fp8_rows_ok(d_q, q_stride, cols) || !ptr_ok(d_scales, 4))) return RS_ERR_INVALID_ARG;
    if (d_rstd && !ptr_ok(d_rstd, 4)) return RS_ERR_INVALID_ARG;
    const bool vec = ptr_ok(d_weight, 16) && rows16(d_x, x_stride, z) &&
                     (!d_residual || rows16(d_residual, residual_stride, z)) &&
                     (!d_sum || rows16(d_sum, sum_stride, z)) && (!d_y || rows16(d_y, y_stride, z));
    NormArgs a{rows, cols, d_x, x_stride, d_residual, residual_stride, d_weight, eps, 1.0f / float(cols), d_sum,
               sum_stride, d_y, y_stride, d_q, q_stride, d_scales, d_rstd};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        bool taken = false;
        const cudaError_t e = vec ? fwd_exact<T>(a, s, taken) : cudaSuccess;
        return taken ? e : vec ? fwd_width<T, kVec>(a, s) : fwd_width<T, kAny>(a, s);
    });
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

size_t rs_rms_norm_bwd_workspace_size(int32_t rows, int32_t cols) {
    if (rows < 0 || cols < 1 || cols > RS_NORM_MAX_COLS) return 0;
    return size_t(rs::bwd_blocks(rows, cols)) * cols * sizeof(float);
}

int rs_rms_norm_bwd(int32_t rows, int32_t cols, int32_t dtype, const void* d_s, size_t s_stride,
                    const float* d_weight, const float* d_rstd, const void* d_dL_dy, size_t dy_stride,
                    const void* d_dL_dsum, size_t dsum_stride, void* d_dL_dx, size_t dx_stride, float* d_dL_dweight,
                    void* d_workspace, size_t workspace_bytes, void* stream) {
    using namespace rs;
    if (rows < 0 || cols < 1 || cols > RS_NORM_MAX_COLS || !dtype_ok(dtype)) return RS_ERR_INVALID_ARG;
    if (d_dL_dweight && !ptr_ok(d_dL_dweight, 4)) return RS_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (!d_dL_dweight) return RS_OK;
        return cudaMemsetAsync(d_dL_dweight, 0, size_t(cols) * 4, s) == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    }
    const size_t z = dtype_size(dtype);
    if (!matrix_ok(d_s, s_stride, cols, dtype) || !matrix_ok(d_dL_dy, dy_stride, cols, dtype) ||
        !matrix_ok(d_dL_dx, dx_stride, cols, dtype) || !ptr_ok(d_weight, 4) || !ptr_ok(d_rstd, 4))
        return RS_ERR_INVALID_ARG;
    if (d_dL_dsum && !matrix_ok(d_dL_dsum, dsum_stride, cols, dtype)) return RS_ERR_INVALID_ARG;
    if ((d_dL_dx == d_dL_dy && dx_stride != dy_stride) || (d_dL_dx == d_dL_dsum && dx_stride != dsum_stride))
        return RS_ERR_INVALID_ARG;
    if (d_dL_dweight) {
        if (!ptr_ok(d_workspace, 16)) return RS_ERR_INVALID_ARG;
        if (workspace_bytes < rs_rms_norm_bwd_workspace_size(rows, cols)) return RS_ERR_WORKSPACE;
    }
    const bool vec = ptr_ok(d_weight, 16) && rows16(d_s, s_stride, z) && rows16(d_dL_dy, dy_stride, z) &&
                     rows16(d_dL_dx, dx_stride, z) &&
                     (!d_dL_dsum || rows16(d_dL_dsum, dsum_stride, z));
    NormBwdArgs a{rows, cols, d_s, s_stride, d_weight, d_rstd, d_dL_dy, dy_stride, d_dL_dsum, dsum_stride, d_dL_dx,
                  dx_stride, d_dL_dweight ? static_cast<float*>(d_workspace) : nullptr, 1.0f / float(cols)};
    cudaError_t e = with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        return vec ? bwd_width<T, true>(a, s) : bwd_width<T, false>(a, s);
    });
    if (e == cudaSuccess && d_dL_dweight)
        e = pdl_launch(k_column_sums, ceil_div(cols, 32), 1024, 0, s, static_cast<const float*>(a.part),
                       bwd_blocks(rows, cols), cols, d_dL_dweight);
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
