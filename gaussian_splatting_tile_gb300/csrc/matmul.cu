// Matrix product of two 8-bit matrices with a scale for each block of 128 along the contracted axis.
//
//   out[i][j] = sum_b sa[b][i] sb[b][j] sum_{t in block b} a[i][t] b[j][t]
//
// The scales change with the block, so a block's products are summed by themselves and added, scaled, to the float32
// total.
#include "wide.cuh"

namespace rs {
namespace {

__device__ unsigned int g_matmul_error;  // set when a bounded wait gave up

struct MatmulArgs {
    int m, n, k;
    const uint8_t* a; size_t as;
    const float* sa;
    const uint8_t* b; size_t bs;
    const float* sb;
    int b_rows;                 // rows of b that share a scale: 1 or 128
    int relu;
    void* out; size_t os;
};

__device__ __forceinline__ float e4m3_to_f(uint8_t x) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(x)));
    return __half2float(__ushort_as_half(uint16_t(h)));
}

template <typename T>
__global__ void __launch_bounds__(256) k_matmul_fp8(MatmulArgs g) {
    RS_PDL_ENTER();
    __shared__ float sa[64][33], sb[64][33];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long i0 = (long long)blockIdx.x * 64, j0 = (long long)blockIdx.y * 64;
    float total[4][4] = {};
    for (int b = 0; b * kBlock < g.k; ++b) {
        float part[4][4] = {};
        for (int t0 = b * kBlock; t0 < min(g.k, (b + 1) * kBlock); t0 += 32) {
            for (int e = threadIdx.x; e < 64 * 32; e += 256) {
                const int r = e >> 5, t = t0 + (e & 31);
                sa[r][e & 31] = i0 + r < g.m && t < g.k ? e4m3_to_f(g.a[(i0 + r) * g.as + t]) : 0.f;
                sb[r][e & 31] = j0 + r < g.n && t < g.k ? e4m3_to_f(g.b[(j0 + r) * g.bs + t]) : 0.f;
            }
            __syncthreads();
            for (int t = 0; t < 32; ++t)
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x) part[y][x] = fmaf(sa[ty + 16 * y][t], sb[tx + 16 * x][t], part[y][x]);
            __syncthreads();
        }
        const int per = g.b_rows == 1 ? g.n : (g.n + kBlock - 1) / kBlock;
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const long long i = i0 + ty + 16 * y, j = j0 + tx + 16 * x;
                if (i < g.m && j < g.n)
                    total[y][x] = fmaf(g.sa[size_t(b) * g.m + i] * g.sb[size_t(b) * per + j / g.b_rows], part[y][x],
                                       total[y][x]);
            }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const long long i = i0 + ty + 16 * y, j = j0 + tx + 16 * x;
            float v = total[y][x];
            if (g.relu && v < 0.f) v = 0.f;
            if (i < g.m && j < g.n) static_cast<T*>(g.out)[i * g.os + j] = from_f<T>(v);
        }
}

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

size_t rs_matmul_fp8_workspace_size(int32_t, int32_t, int32_t) { return 0; }

int rs_matmul_fp8(int32_t m, int32_t n, int32_t k, const uint8_t* d_a, size_t a_stride, const float* d_a_scales,
                  const uint8_t* d_b, size_t b_stride, const float* d_b_scales, int32_t b_scale_rows, int32_t relu,
                  int32_t out_dtype, void* d_out, size_t out_stride, void* d_workspace, size_t workspace_bytes,
                  void* stream) {
    using namespace rs;
    if (m < 0 || n < 0 || k < 0 || !dtype_ok(out_dtype) || (b_scale_rows != 1 && b_scale_rows != kBlock))
        return RS_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return RS_OK;
    if (!ptr_ok(d_out, dtype_size(out_dtype)) || out_stride < size_t(n)) return RS_ERR_INVALID_ARG;
    if (k > 0 && (!fp8_rows_ok(d_a, a_stride, k) || !fp8_rows_ok(d_b, b_stride, k) || !ptr_ok(d_a_scales, 4) ||
                  !ptr_ok(d_b_scales, 4)))
        return RS_ERR_INVALID_ARG;
    const size_t need = rs_matmul_fp8_workspace_size(m, n, k);
    if (need > 0 && !ptr_ok(d_workspace, 16)) return RS_ERR_INVALID_ARG;
    if (workspace_bytes < need) return RS_ERR_WORKSPACE;
    MatmulArgs g{m, n, k, d_a, a_stride, d_a_scales, d_b, b_stride, d_b_scales, b_scale_rows, relu, d_out, out_stride};
    const cudaError_t e = with_dtype(out_dtype, [&](auto v) {
        return pdl_launch(k_matmul_fp8<decltype(v)>, dim3(ceil_div(m, 64), ceil_div(n, 64)), 256, 0,
                          static_cast<cudaStream_t>(stream), g);
    });
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
