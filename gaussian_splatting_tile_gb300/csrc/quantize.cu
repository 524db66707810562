// 8-bit forms of a matrix: blocks of 128 along a row, blocks of 128 rows (written transposed), or 128 x 128.
//
// One thread block takes a 128 x 128 tile, so that every scale is settled inside it and one read of x gives both
// forms.  A thread holds 8 rows x 8 columns: a row's maximum is a shuffle over the 16 threads beside it, a column's goes
// through shared memory over the 16 above and below.  Bound by memory: 2 or 4 bytes in, one or two out.
#include "wide.cuh"

namespace rs {
namespace {

struct QuantArgs {
    int rows, cols;
    const void* x; size_t xs;
    const void* relu; size_t relus;
    uint8_t* q; size_t qs;
    float* scales;
    uint8_t* qt; size_t qts;
    float* scales_t;
    int ctiles, rtiles;
};

template <typename T, bool VEC, bool BLOCKS>
__global__ void __launch_bounds__(256) k_quantize(QuantArgs a) {
    RS_PDL_ENTER();
    __shared__ float cmax[16][kBlock + 4];
    __shared__ __align__(16) uint8_t tile[kBlock][kBlock + 16];  // the transposed bytes
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int ct = blockIdx.x % a.ctiles, rt = blockIdx.x / a.ctiles;  // neighbours share the rows
    const int c0 = ct * kBlock, c = c0 + tx * 8;
    const long long r0 = (long long)rt * kBlock, r = r0 + ty * 8;
    const int left = a.cols - c;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool in = r + i < a.rows;
        load8<T, VEC>(static_cast<const T*>(a.x) + (in ? r + i : 0) * a.xs + c, in ? left : 0, v[i]);
        if (a.relu) {
            float u[8];
            load8<T, VEC>(static_cast<const T*>(a.relu) + (in ? r + i : 0) * a.relus + c, in ? left : 0, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = u[j] <= 0.f ? 0.f : v[i][j];
        }
    }
    if constexpr (BLOCKS) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_abs8(v[i], m);
        m = group_max<32>(m);
        if ((threadIdx.x & 31) == 0) cmax[0][threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, cmax[0][i]);
        float scale, inv;
        block_scale(m, scale, inv);
        if (threadIdx.x == 0) {
            if (a.q) a.scales[size_t(ct) * a.rtiles + rt] = scale;
            if (a.qt) a.scales_t[size_t(rt) * a.ctiles + ct] = scale;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= inv;
            if (a.q && r + i < a.rows && left > 0) store8_e4m3(a.q + (r + i) * a.qs + c, left, v[i], 1.f);
        }
    } else {
        if (a.q) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float scale, inv;
                block_scale(group_max<16>(max_abs8(v[i], 0.f)), scale, inv);
                if (r + i < a.rows && left > 0) {
                    store8_e4m3(a.q + (r + i) * a.qs + c, left, v[i], inv);
                    if (tx == 0) a.scales[size_t(ct) * a.rows + r + i] = scale;
                }
            }
        }
        if (!a.qt) return;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i][j]));
            cmax[ty][tx * 8 + j] = m;
        }
        __syncthreads();
        if (threadIdx.x < kBlock) {
            float m = 0.f, scale, inv;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, cmax[i][threadIdx.x]);
            block_scale(m, scale, inv);
            if (c0 + int(threadIdx.x) < a.cols) a.scales_t[size_t(rt) * a.cols + c0 + threadIdx.x] = scale;
            cmax[0][threadIdx.x] = inv;  // this column of row 0 is read by this thread alone
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float inv = cmax[0][tx * 8 + j];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i][j] *= inv;
        }
    }
    if (!a.qt) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t lo = e4m3x4(v[0][j], v[1][j], v[2][j], v[3][j]);
        const uint32_t hi = e4m3x4(v[4][j], v[5][j], v[6][j], v[7][j]);
        *reinterpret_cast<uint2*>(&tile[tx * 8 + j][ty * 8]) = make_uint2(lo, hi);
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int tc = p * 32 + int(threadIdx.x >> 3), tr = int(threadIdx.x & 7) * 16;
        if (c0 + tc >= a.cols || r0 + tr >= a.rows) continue;
        uint8_t* o = a.qt + size_t(c0 + tc) * a.qts + r0 + tr;
        const long long rest = a.rows - (r0 + tr);
        if (rest >= 16) {
            *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(&tile[tc][tr]);
        } else {
            for (int i = 0; i < rest; ++i) o[i] = tile[tc][tr + i];
        }
    }
}

int quantize(QuantArgs a, int32_t dtype, bool blocks, cudaStream_t s) {
    if (a.rows < 0 || a.cols < 0 || !dtype_ok(dtype)) return RS_ERR_INVALID_ARG;
    if ((a.q == nullptr) != (a.scales == nullptr) || (a.qt == nullptr) != (a.scales_t == nullptr))
        return RS_ERR_INVALID_ARG;
    if (a.rows == 0 || a.cols == 0) return RS_OK;
    if (!a.q && !a.qt) return RS_ERR_INVALID_ARG;
    const size_t z = dtype_size(dtype);
    if (!ptr_ok(a.x, z) || a.xs < size_t(a.cols)) return RS_ERR_INVALID_ARG;
    if (a.relu && (!ptr_ok(a.relu, z) || a.relus < size_t(a.cols))) return RS_ERR_INVALID_ARG;
    if (a.q && (!fp8_rows_ok(a.q, a.qs, a.cols) || !ptr_ok(a.scales, 4))) return RS_ERR_INVALID_ARG;
    if (a.qt && (!fp8_rows_ok(a.qt, a.qts, a.rows) || !ptr_ok(a.scales_t, 4))) return RS_ERR_INVALID_ARG;
    a.ctiles = ceil_div(a.cols, kBlock);
    a.rtiles = ceil_div(a.rows, kBlock);
    if ((long long)a.ctiles * a.rtiles > 0x7fffffffLL) return RS_ERR_INVALID_ARG;
    const bool vec = rows16(a.x, a.xs, z) && (!a.relu || rows16(a.relu, a.relus, z));
    const cudaError_t e = with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        const unsigned g = unsigned(a.ctiles) * a.rtiles;
        if (blocks)
            return vec ? pdl_launch(k_quantize<T, true, true>, g, 256, 0, s, a)
                       : pdl_launch(k_quantize<T, false, true>, g, 256, 0, s, a);
        return vec ? pdl_launch(k_quantize<T, true, false>, g, 256, 0, s, a)
                   : pdl_launch(k_quantize<T, false, false>, g, 256, 0, s, a);
    });
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // namespace
}  // namespace rs

extern "C" {

int rs_quantize_fp8(int32_t rows, int32_t cols, int32_t dtype, const void* d_x, size_t x_stride, const void* d_relu,
                    size_t relu_stride, uint8_t* d_q, size_t q_stride, float* d_scales, uint8_t* d_qt,
                    size_t qt_stride, float* d_scales_t, void* stream) {
    return rs::quantize({rows, cols, d_x, x_stride, d_relu, relu_stride, d_q, q_stride, d_scales, d_qt, qt_stride,
                         d_scales_t, 0, 0}, dtype, false, static_cast<cudaStream_t>(stream));
}

int rs_quantize_fp8_blocks(int32_t rows, int32_t cols, int32_t dtype, const void* d_x, size_t x_stride, uint8_t* d_q,
                           size_t q_stride, float* d_scales, uint8_t* d_qt, size_t qt_stride, float* d_scales_t,
                           void* stream) {
    return rs::quantize({rows, cols, d_x, x_stride, nullptr, 0, d_q, q_stride, d_scales, d_qt, qt_stride, d_scales_t,
                         0, 0}, dtype, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
