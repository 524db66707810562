// Shared by the kernels of the wide appearance networks (norm.cu, quantize.cu, matmul.cu, clip.cu): element
// types, runs of eight values, and the 8-bit form with a scale for each block of 128.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "rs_internal.cuh"

namespace rs {

constexpr int kBlock = RS_FP8_BLOCK;
constexpr int kSms = 152;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight consecutive values at `p`, of which the first `left` exist (the others read as zero).  VEC: p is aligned to
// 16 bytes; a whole run is then one or two 16-byte accesses.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int left, float (&v)[8]) {
    if (VEC && left >= 8) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            const T* h = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_f(h[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f(p[i]) : 0.f;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int left, const float (&v)[8]) {
    if (VEC && left >= 8) {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint4 w;
            T* h = reinterpret_cast<T*>(&w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = from_f<T>(v[i]);
            *reinterpret_cast<uint4*>(p) = w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = from_f<T>(v[i]);
}

// Four floats as e4m3 bytes, lowest first (round to nearest even; finite values past 448 become 448, NaN stays).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return uint32_t(lo) | (uint32_t(hi) << 16);
}

// Eight scaled values as bytes.  A row starts on a 16-byte boundary and runs of eight on multiples of 8.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int left, const float (&v)[8], float inv) {
    const uint32_t lo = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    const uint32_t hi = e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    if (left >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = uint8_t((i < 4 ? lo : hi) >> (8 * (i & 3)));
}

// A block's scale and the factor its values are multiplied by, from its largest magnitude.  Both are correctly rounded
// quotients: that makes the 8-bit form a function of the values alone, equal on every path.
__device__ __forceinline__ void block_scale(float amax, float& scale, float& inv) {
    const float a = fmaxf(amax, 7.888609052210118e-31f);  // 2^-100: a block of zeros, and no overflow of 448 / a
    scale = __fdiv_rn(a, 448.f);
    inv = __fdiv_rn(448.f, a);
}

__device__ __forceinline__ float max_abs8(const float (&v)[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

template <int W>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <int W>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The gradient norm from its partial sums of squares, the same bits in every block; all 256 threads call it.
__device__ __forceinline__ float norm_of_parts(const float* part, int parts) {
    __shared__ double sm[8];
    double v = 0.0;
    for (int i = threadIdx.x; i < parts; i += 256) v += double(part[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += sm[i];
    return sqrtf(float(v));
}

// min(1, max_norm / (norm + 1e-6)), a NaN norm's NaN kept.
__device__ __forceinline__ float clip_factor(float max_norm, float norm) {
    const float c = max_norm / (norm + 1e-6f);
    return c > 1.f ? 1.f : c;
}

// ---- host side
inline bool dtype_ok(int32_t t) { return t == RS_F32 || t == RS_F16 || t == RS_BF16; }
inline size_t dtype_size(int32_t t) { return t == RS_F32 ? 4 : 2; }
inline bool ptr_ok(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
// rows of 8 values can be moved with 16-byte accesses
inline bool rows16(const void* p, size_t stride, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0;
}
inline bool fp8_rows_ok(const void* p, size_t stride, int32_t cols) {
    return ptr_ok(p, 16) && stride % 16 == 0 && stride >= size_t(cols);
}
inline int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

// Calls f with a value of the element type.
template <typename F>
auto with_dtype(int32_t t, F&& f) {
    if (t == RS_F32) return f(float());
    if (t == RS_F16) return f(__half());
    return f(__nv_bfloat16());
}

}  // namespace rs
