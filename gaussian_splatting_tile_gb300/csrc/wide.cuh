// Shared by the kernels of the wide appearance networks (norm.cu, quantize.cu, matmul.cu, clip.cu): element
// types, runs of eight values, and the 8-bit form with a scale for each block of 128.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "matmul_plan.h"
#include "rs_internal.cuh"

namespace rs {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight consecutive values as they are stored, of which the first `left` exist (the others read as zero).  VEC: the
// place is aligned to 16 bytes, and a whole run is one or two 16-byte accesses; else a run of 16-bit values is read
// as aligned words where its neighbours on both sides exist (`inner`).  16-bit types stay packed in four registers,
// where a maximum of magnitudes is exact, and are widened where they are used.
template <typename T>
struct Run8 {
    float v[8];
    __device__ __forceinline__ float2 pair(int p) const { return make_float2(v[2 * p], v[2 * p + 1]); }
    template <bool VEC>
    __device__ __forceinline__ void load(const T* p, int left, bool = false) {
        if (VEC && left >= 8) {
            const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.f;
        }
    }
    // zero where u <= 0
    __device__ __forceinline__ void mask(const Run8& u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = u.v[i] <= 0.f ? 0.f : v[i];
    }
    // m = max(m, |values|), pair by pair
    struct Max { float x = 0.f, y = 0.f; };
    __device__ __forceinline__ void max_into(Max& m, int p) const {
        m.x = fmaxf(m.x, fabsf(v[2 * p]));
        m.y = fmaxf(m.y, fabsf(v[2 * p + 1]));
    }
    static __device__ __forceinline__ float2 wide(const Max& m) { return make_float2(m.x, m.y); }
};

template <typename T, typename T2>
struct PackedRun8 {
    uint4 w;
    __device__ __forceinline__ uint32_t word(int p) const { return p == 0 ? w.x : p == 1 ? w.y : p == 2 ? w.z : w.w; }
    __device__ __forceinline__ float2 pair(int p) const {
        const uint32_t x = word(p);
        const T2 h = *reinterpret_cast<const T2*>(&x);
        return make_float2(to_f(h.x), to_f(h.y));
    }
    template <bool VEC>
    __device__ __forceinline__ void load(const T* p, int left, bool inner = false) {
        if (VEC && left >= 8) {
            w = *reinterpret_cast<const uint4*>(p);
        } else if (inner && left > 8) {
            // five aligned words hold the run; half a word too many where it starts on one
            const uint32_t shift = reinterpret_cast<uintptr_t>(p) & 2 ? 16 : 0;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
            const uint32_t a = q[0], b = q[1], c = q[2], d = q[3], e = shift ? q[4] : 0u;
            w = make_uint4(__funnelshift_r(a, b, shift), __funnelshift_r(b, c, shift), __funnelshift_r(c, d, shift),
                           __funnelshift_r(d, e, shift));
        } else {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = i < left ? q[i] : 0;
            w = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
    }
    static __device__ __forceinline__ uint32_t kept(uint32_t x, uint32_t u) {
        return x & ~__hle2_mask(*reinterpret_cast<const T2*>(&u), T2{T(0.f), T(0.f)});
    }
    __device__ __forceinline__ void mask(const PackedRun8& u) {
        w = make_uint4(kept(w.x, u.w.x), kept(w.y, u.w.y), kept(w.z, u.w.z), kept(w.w, u.w.w));
    }
    struct Max { T2 h = {T(0.f), T(0.f)}; };
    __device__ __forceinline__ void max_into(Max& m, int p) const {
        const uint32_t x = word(p) & 0x7fff7fffu;
        m.h = __hmax2(m.h, *reinterpret_cast<const T2*>(&x));
    }
    static __device__ __forceinline__ float2 wide(const Max& m) { return make_float2(to_f(m.h.x), to_f(m.h.y)); }
};
template <> struct Run8<__half> : PackedRun8<__half, __half2> {};
template <> struct Run8<__nv_bfloat16> : PackedRun8<__nv_bfloat16, __nv_bfloat162> {};

// Four floats as e4m3 bytes, lowest first (round to nearest even; finite values past 448 become 448, NaN stays).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return uint32_t(lo) | (uint32_t(hi) << 16);
}

// The same as floats.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int left, float (&v)[8], bool inner = false) {
    Run8<T> r;
    r.template load<VEC>(p, left, inner);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 w = r.pair(i);
        v[2 * i] = w.x;
        v[2 * i + 1] = w.y;
    }
}

__device__ __forceinline__ uint32_t pack_pair(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int left, const float (&v)[8]) {
    if (VEC && left >= 8) {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(pack_pair(v[0], v[1], T()), pack_pair(v[2], v[3], T()),
                                                      pack_pair(v[4], v[5], T()), pack_pair(v[6], v[7], T()));
        }
        return;
    }
    if constexpr (!VEC && sizeof(T) == 2) {
        if (left >= 8) {  // whole words, with one value before and one after them where the run does not start on one
            uint32_t* q = reinterpret_cast<uint32_t*>((reinterpret_cast<uintptr_t>(p) + 3) & ~uintptr_t(3));
            if (reinterpret_cast<uintptr_t>(p) & 2) {
                p[0] = from_f<T>(v[0]);
#pragma unroll
                for (int i = 0; i < 3; ++i) q[i] = pack_pair(v[2 * i + 1], v[2 * i + 2], T());
                p[7] = from_f<T>(v[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = pack_pair(v[2 * i], v[2 * i + 1], T());
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = from_f<T>(v[i]);
}

// Up to eight bytes of a row.  A row starts on a 16-byte boundary and runs of eight on multiples of 8.
__device__ __forceinline__ void store8_bytes(uint8_t* p, int left, uint32_t lo, uint32_t hi) {
    if (left >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = uint8_t((i < 4 ? lo : hi) >> (8 * (i & 3)));
}

// Eight values, scaled, as bytes.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int left, const float (&v)[8], float inv) {
    store8_bytes(p, left, e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                 e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}
template <typename T>
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int left, const Run8<T>& v, float inv) {
    const float2 a = v.pair(0), b = v.pair(1), c = v.pair(2), d = v.pair(3);
    store8_bytes(p, left, e4m3x4(a.x * inv, a.y * inv, b.x * inv, b.y * inv),
                 e4m3x4(c.x * inv, c.y * inv, d.x * inv, d.y * inv));
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

template <typename T>
__device__ __forceinline__ float max_abs8(const Run8<T>& v) {
    typename Run8<T>::Max m;
#pragma unroll
    for (int p = 0; p < 4; ++p) v.max_into(m, p);
    const float2 w = Run8<T>::wide(m);
    return fmaxf(w.x, w.y);
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

// The gradient norm from its partial sums of squares, the same bits in every block; all 256 threads call it.  In
// float32: the sums are positive and the chains short, and in float64 this alone took 27 us of a step over 59 M
// parameters.
__device__ __forceinline__ float norm_of_parts(const float* part, int parts) {
    __shared__ float sm[8];
    float v = 0.f;
    for (int i = threadIdx.x; i < parts; i += 256) v += part[i];
    v = group_sum<32>(v);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += sm[i];
    return sqrtf(v);
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

// Calls f with a value of the element type.
template <typename F>
auto with_dtype(int32_t t, F&& f) {
    if (t == RS_F32) return f(float());
    if (t == RS_F16) return f(__half());
    return f(__nv_bfloat16());
}

}  // namespace rs
