// 8-bit forms of a matrix: blocks of 128 along a row, blocks of 128 rows (written transposed), or 128 x 128.
//
// One thread block takes a 128 x 128 tile, so that every scale is settled inside it and one read of x gives both
// forms.  A thread holds 8 rows x 8 columns: a row's maximum is a shuffle over the 16 threads beside it, a column's
// goes through shared memory over the 16 above and below.  Bound by memory: 2 or 4 bytes in, one or two out.
//
// Measured: 160,000 x 512 bf16 both forms 60 us (5.4 TB/s), through a relu 85 us (5.8 TB/s), float32 5.9 TB/s; 128 x 128
// forms both ways round of 8192 x 8192 float32 68 us (5.9 TB/s), bf16 51 us (5.2 TB/s), of 2048 x 2048 10 us, the launch.
// Through a relu kept in 8 bits 160,000 x 512 bf16 67 us (6.1 TB/s); 80,000 x 1001, rows between words, 120 us (3.4 TB/s).
#include "wide.cuh"

namespace rs {
namespace {

struct QuantArgs {
    int rows, cols;
    const void* x; size_t xs;
    const void* relu; size_t relus;   // of x's type, or (relu8) in 8 bits
    uint8_t* q; size_t qs;
    float* scales;
    uint8_t* qt; size_t qts;
    float* scales_t;
    int ctiles, rtiles;
};

// Where the transposed tile keeps the eight bytes of column c, rows 8 u to 8 u + 7: the sixteen threads that write
// the same u of sixteen columns eight apart, and the eight that read a column's sixteen-byte words, all hit different
// banks.
__device__ __forceinline__ int tile_unit(int c, int u) { return c * 16 + (u ^ ((c >> 3) & 15)); }

// The 8 x 8 values of one thread, scaled by column (inv[j]), to the transposed bytes.
template <typename T>
__device__ __forceinline__ void store_transposed(const QuantArgs& a, const Run8<T> (&v)[8], const float (&inv)[8],
                                                 uint2* tile, int tx, int ty, int c0, long long r0) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 w = v[i].pair(j / 2);
            x[i] = w.x * inv[j];
            y[i] = w.y * inv[j + 1];
        }
        uint2* at = tile + tile_unit(tx * 8 + j, ty);  // the next column is 16 units on
        at[0] = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
        at[16] = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int tc = p * 32 + int(threadIdx.x >> 3), k = int(threadIdx.x & 7), tr = k * 16;
        if (c0 + tc >= a.cols || r0 + tr >= a.rows) continue;
        uint8_t* o = a.qt + size_t(c0 + tc) * a.qts + r0 + tr;
        const uint2 lo = tile[tile_unit(tc, 2 * k)], hi = tile[tile_unit(tc, 2 * k + 1)];
        const uint4 w = make_uint4(lo.x, lo.y, hi.x, hi.y);
        const long long rest = a.rows - (r0 + tr);
        if (rest >= 16) {
            *reinterpret_cast<uint4*>(o) = w;
        } else {
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < rest) o[i] = uint8_t(ws[i >> 2] >> (8 * (i & 3)));
        }
    }
}

// 16-bit values leave registers for three blocks an SM; with a mask beside x two, so that both tiles are in flight at
// once.
enum Form { kRowsCols, kRowsColsRelu, kRowsColsRelu8, kBlocks };
// FULL: 16-byte rows, and no tile ends inside its columns.
template <typename T, bool VEC, bool FULL, Form FORM>
__global__ void __launch_bounds__(256, sizeof(T) == 4 || FORM == kRowsColsRelu || FORM == kRowsColsRelu8 ? 2 : 3)
    k_quantize(QuantArgs a) {
    constexpr bool BLOCKS = FORM == kBlocks;
    RS_PDL_ENTER();
    __shared__ float cmax[16][kBlock];
    __shared__ __align__(16) uint2 tile[kBlock * 16];  // the transposed bytes
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int ct = blockIdx.x % a.ctiles, rt = blockIdx.x / a.ctiles;  // neighbours share the rows
    const int c0 = ct * kBlock, c = c0 + tx * 8;
    const long long r0 = (long long)rt * kBlock, r = r0 + ty * 8;
    // through a checkpoint, 16-byte rows come in whole runs of eight (80,000 x 1000 bf16: 70 us, 88 with ragged ones)
    const int left = FULL ? 8 : FORM == kRowsColsRelu8 && VEC ? (c < a.cols ? 8 : 0) : a.cols - c;
    Run8<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool in = r + i < a.rows;
        const T* p = static_cast<const T*>(a.x) + (in ? r + i : 0) * a.xs + c;
        if constexpr (FORM == kRowsColsRelu8 && !VEC) v[i].load_words(p, in ? left : 0);
        else v[i].template load<VEC>(p, in ? left : 0, c > 0);
    }
    if constexpr (FORM == kRowsColsRelu) {
        Run8<T> u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = r + i < a.rows;
            const T* p = static_cast<const T*>(a.relu) + (in ? r + i : 0) * a.relus + c;
            u[i].template load<VEC>(p, in ? left : 0, c > 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].mask(u[i]);
    }
    if constexpr (FORM == kRowsColsRelu8) {
        Bytes8 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = r + i < a.rows;
            u[i].load(static_cast<const uint8_t*>(a.relu) + (in ? r + i : 0) * a.relus + c, in ? left : 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].mask(u[i]);
    }
    if constexpr (BLOCKS) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, max_abs8(v[i]));
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
        if (a.q) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r + i < a.rows && left > 0) store8_e4m3(a.q + (r + i) * a.qs + c, left, v[i], inv);
        }
        const float invs[8] = {inv, inv, inv, inv, inv, inv, inv, inv};
        if (a.qt) store_transposed(a, v, invs, tile, tx, ty, c0, r0);
    } else {
        if (a.q) {
            // The eight rows' maxima over the sixteen threads beside each other: every exchange halves the rows that
            // a thread goes on with, so that thread tx ends with row (tx >> 1 & 7) and forms that row's two quotients
            // alone.
            float m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = max_abs8(v[i]);
#pragma unroll
            for (int o = 8, n = 4; n; o >>= 1, n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const bool upper = tx & o;
                    const float other = __shfl_xor_sync(0xffffffffu, upper ? m[i] : m[i + n], o);
                    m[i] = fmaxf(upper ? m[i + n] : m[i], other);
                }
            float scale, inv;
            block_scale(fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1)), scale, inv);
            const int mine = (tx & 8 ? 4 : 0) + (tx & 4 ? 2 : 0) + (tx & 2 ? 1 : 0);
            if (!(tx & 1) && r + mine < a.rows) a.scales[size_t(ct) * a.rows + r + mine] = scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int from = (i & 4 ? 8 : 0) + (i & 2 ? 4 : 0) + (i & 1 ? 2 : 0);
                const float k = __shfl_sync(0xffffffffu, inv, from, 16);
                if (r + i < a.rows && left > 0) store8_e4m3(a.q + (r + i) * a.qs + c, left, v[i], k);
            }
        }
        if (!a.qt) return;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            typename Run8<T>::Max m;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i].max_into(m, p);
            *reinterpret_cast<float2*>(&cmax[ty][tx * 8 + 2 * p]) = Run8<T>::wide(m);
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
        float invs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) invs[j] = cmax[0][tx * 8 + j];
        store_transposed(a, v, invs, tile, tx, ty, c0, r0);
    }
}

// The transposed form of a checkpoint: 128 rows x 64 columns a block, a thread 8 x 8 values, which are a byte times
// their row's scale.  They stay bytes and are widened twice, for the columns' maxima and for their new bytes: that leaves
// registers for ten blocks an SM, which load, compute and store in turn.  One byte in, one out, and nearly enough
// instructions to fill that time: 250,000 x 512 48.5 us (5.4 TB/s); with tiles of 128 columns 56, kept wide 63.
constexpr int kHalf = kBlock / 2;

__global__ void __launch_bounds__(128, 10) k_transpose(QuantArgs a, bool vec) {
    RS_PDL_ENTER();
    __shared__ __align__(8) float cmax[4][kHalf];
    __shared__ __align__(16) uint2 tile[kHalf * 16];  // eight bytes of column c, rows 8 u on: at 16 c + (u ^ 2 (c / 8))
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int ct = blockIdx.x % a.ctiles, rt = blockIdx.x / a.ctiles;
    const int c0 = ct * kHalf, c = c0 + tx * 8;
    const long long r0 = (long long)rt * kBlock, r = r0 + ty * 8;
    const int left = a.cols - c;
    Bytes8 v[8];
    float scale[8];
    const uint8_t* from = static_cast<const uint8_t*>(a.x) + r * a.xs + c;
    const float* sc = a.scales + size_t(ct >> 1) * a.rows + r;
    if (r0 + kBlock <= a.rows && c0 + kHalf <= a.cols && a.rows % 4 == 0 && vec) {  // nothing to ask (asking: 56 us)
#pragma unroll
        for (int i = 0; i < 8; ++i, from += a.xs) v[i].load(from, 8);
        const float4 lo = reinterpret_cast<const float4*>(sc)[0], hi = reinterpret_cast<const float4*>(sc)[1];
        scale[0] = lo.x, scale[1] = lo.y, scale[2] = lo.z, scale[3] = lo.w;
        scale[4] = hi.x, scale[5] = hi.y, scale[6] = hi.z, scale[7] = hi.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i, from += a.xs) {
            const bool in = r + i < a.rows;
            v[i].load(from, in ? left : 0);
            scale[i] = in ? sc[i] : 0.f;
        }
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float2 m = f2(0.f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 f = f2_mul(v[i].pair(p), f2(scale[i])), g = f2_mul(v[i + 1].pair(p), f2(scale[i + 1]));
            m = make_float2(max3(m.x, fabsf(f.x), fabsf(g.x)), max3(m.y, fabsf(f.y), fabsf(g.y)));
        }
#pragma unroll
        for (int o = 8; o < 32; o *= 2) {
            m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, o));
            m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
        }
        if (!(ty & 3)) *reinterpret_cast<float2*>(&cmax[ty >> 2][tx * 8 + 2 * p]) = m;
    }
    __syncthreads();
    if (threadIdx.x < kHalf) {
        float out, inv;
        const float m = fmaxf(fmaxf(cmax[0][threadIdx.x], cmax[1][threadIdx.x]),
                              fmaxf(cmax[2][threadIdx.x], cmax[3][threadIdx.x]));
        block_scale(m, out, inv);
        if (c0 + int(threadIdx.x) < a.cols) a.scales_t[size_t(rt) * a.cols + c0 + threadIdx.x] = out;
        cmax[0][threadIdx.x] = inv;  // this column of row 0 is read by this thread alone
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(v[i].w.x), "+r"(v[i].w.y));  // widened anew, not kept wide
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const float2 inv = *reinterpret_cast<const float2*>(&cmax[0][tx * 8 + 2 * p]);
        float2 f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f2_mul(f2_mul(v[i].pair(p), f2(scale[i])), inv);
        uint2* at = tile + (tx * 8 + 2 * p) * 16 + (ty ^ 2 * tx);
        at[0] = make_uint2(e4m3x4(f[0].x, f[1].x, f[2].x, f[3].x), e4m3x4(f[4].x, f[5].x, f[6].x, f[7].x));
        at[16] = make_uint2(e4m3x4(f[0].y, f[1].y, f[2].y, f[3].y), e4m3x4(f[4].y, f[5].y, f[6].y, f[7].y));
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int tc = p * 16 + ty, k = tx, tr = k * 16;
        if (c0 + tc >= a.cols || r0 + tr >= a.rows) continue;
        uint8_t* o = a.qt + size_t(c0 + tc) * a.qts + r0 + tr;
        const uint4 w = *reinterpret_cast<const uint4*>(tile + tc * 16 + (2 * k ^ 2 * (tc >> 3)));
        const long long rest = a.rows - (r0 + tr);
        if (rest >= 16) {
            *reinterpret_cast<uint4*>(o) = w;
        } else {
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < rest) o[i] = uint8_t(ws[i >> 2] >> (8 * (i & 3)));
        }
    }
}

int quantize(QuantArgs a, int32_t dtype, bool blocks, cudaStream_t s, bool relu8 = false) {
    if (a.rows < 0 || a.cols < 0 || !dtype_ok(dtype)) return RS_ERR_INVALID_ARG;
    if ((a.q == nullptr) != (a.scales == nullptr) || (a.qt == nullptr) != (a.scales_t == nullptr))
        return RS_ERR_INVALID_ARG;
    if (a.rows == 0 || a.cols == 0) return RS_OK;
    if (!a.q && !a.qt) return RS_ERR_INVALID_ARG;
    const size_t z = dtype_size(dtype);
    if (!ptr_ok(a.x, z) || a.xs < size_t(a.cols)) return RS_ERR_INVALID_ARG;
    if (relu8 ? !fp8_rows_ok(a.relu, a.relus, a.cols)
              : a.relu && (!ptr_ok(a.relu, z) || a.relus < size_t(a.cols)))
        return RS_ERR_INVALID_ARG;
    if (a.q && (!fp8_rows_ok(a.q, a.qs, a.cols) || !ptr_ok(a.scales, 4))) return RS_ERR_INVALID_ARG;
    if (a.qt && (!fp8_rows_ok(a.qt, a.qts, a.rows) || !ptr_ok(a.scales_t, 4))) return RS_ERR_INVALID_ARG;
    a.ctiles = ceil_div(a.cols, kBlock);
    a.rtiles = ceil_div(a.rows, kBlock);
    if ((long long)a.ctiles * a.rtiles > 0x7fffffffLL) return RS_ERR_INVALID_ARG;
    const bool vec = rows16(a.x, a.xs, z) && (relu8 ? a.cols % 8 == 0 : !a.relu || rows16(a.relu, a.relus, z));
    const cudaError_t e = with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        const unsigned g = unsigned(a.ctiles) * a.rtiles;
        const auto launch = [&](auto any, auto ragged, auto full) {
            return pdl_launch(!vec ? any : a.cols % kBlock ? ragged : full, g, 256, 0, s, a);
        };
        if (blocks)
            return launch(k_quantize<T, false, false, kBlocks>, k_quantize<T, true, false, kBlocks>,
                          k_quantize<T, true, true, kBlocks>);
        if (relu8)
            return launch(k_quantize<T, false, false, kRowsColsRelu8>, k_quantize<T, true, false, kRowsColsRelu8>,
                          k_quantize<T, true, true, kRowsColsRelu8>);
        if (a.relu)
            return launch(k_quantize<T, false, false, kRowsColsRelu>, k_quantize<T, true, false, kRowsColsRelu>,
                          k_quantize<T, true, true, kRowsColsRelu>);
        return launch(k_quantize<T, false, false, kRowsCols>, k_quantize<T, true, false, kRowsCols>,
                      k_quantize<T, true, true, kRowsCols>);
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

int rs_quantize_fp8_relu8(int32_t rows, int32_t cols, int32_t dtype, const void* d_x, size_t x_stride,
                          const uint8_t* d_relu, size_t relu_stride, uint8_t* d_q, size_t q_stride, float* d_scales,
                          uint8_t* d_qt, size_t qt_stride, float* d_scales_t, void* stream) {
    return rs::quantize({rows, cols, d_x, x_stride, d_relu, relu_stride, d_q, q_stride, d_scales, d_qt, qt_stride,
                         d_scales_t, 0, 0}, dtype, false, static_cast<cudaStream_t>(stream), true);
}

int rs_transpose_fp8(int32_t rows, int32_t cols, const uint8_t* d_q, size_t q_stride, const float* d_scales,
                     uint8_t* d_qt, size_t qt_stride, float* d_scales_t, void* stream) {
    using namespace rs;
    if (rows < 0 || cols < 0) return RS_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return RS_OK;
    if (!fp8_rows_ok(d_q, q_stride, cols) || !ptr_ok(d_scales, 4) || !fp8_rows_ok(d_qt, qt_stride, rows) ||
        !ptr_ok(d_scales_t, 4))
        return RS_ERR_INVALID_ARG;
    const int ctiles = ceil_div(cols, kHalf), rtiles = ceil_div(rows, kBlock);
    if ((long long)ctiles * rtiles > 0x7fffffffLL) return RS_ERR_INVALID_ARG;
    const QuantArgs a{rows, cols, d_q, q_stride, nullptr, 0, nullptr, 0, const_cast<float*>(d_scales), d_qt, qt_stride,
                      d_scales_t, ctiles, rtiles};
    const cudaError_t e = pdl_launch(k_transpose, unsigned(ctiles) * rtiles, 128, 0, static_cast<cudaStream_t>(stream), a,
                                     ptr_ok(d_scales, 16));
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
