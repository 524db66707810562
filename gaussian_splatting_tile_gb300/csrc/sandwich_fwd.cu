#include "sandwich.cuh"

namespace rs {
namespace {

// ---------------------------------------------------------------- forward
// The largest of each of N (a power of two up to 16) values over sixteen neighbouring threads: every exchange halves the
// values that a thread goes on with, so that thread t of the sixteen ends with value t N / 16, in m[0].
template <int N>
__device__ __forceinline__ void max_over_16(float (&m)[N], int t) {
#pragma unroll
    for (int o = 8, n = N / 2; o; o >>= 1, n >>= 1) {
        if (n > 0) {
            const bool upper = t & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float other = __shfl_xor_sync(0xffffffffu, upper ? m[i] : m[i + n], o);
                m[i] = fmaxf(upper ? m[i + n] : m[i], other);
            }
        } else {
            m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        }
    }
}
__host__ __device__ constexpr int power_of_two(int n) { return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : 16; }

// Eight values, scaled, as bytes.
__device__ __forceinline__ void store_e4m3(uint8_t* p, int left, const float2 (&v)[4], float by) {
    float2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f2_mul(v[i], f2(by));
    store8_bytes(p, left, e4m3x4(w[0].x, w[0].y, w[1].x, w[1].y), e4m3x4(w[2].x, w[2].y, w[3].x, w[3].y));
}

// A row stays in registers between its sums, as in the plain norm: TPR threads, RUNS runs of eight values each.  What
// bounds it is memory, once the instructions fit into its time: two runs a thread halve what a thread does once (sums
// over the row, maxima, quotients), and a row of up to 512 values then is a warp's own, without a barrier; arithmetic is
// in pairs; two operands' or three operands' maxima travel together.  That took 250,000 x 512 bf16, gated, operands kept,
// from 384 us (103 instructions a value) to 243 (60; 6.4 TB/s, 94% of the copy's rate).  float32 160,000 x 512 233 us
// (7.1 TB/s); 80,000 x 1000 bf16 199 us (4.9 TB/s: three of a row's 128 runs are empty, and rows of two warps wait for each
// other); 80,000 x 1001, between words, 248 us.  One row costs the call, 10 us, and 3 in a graph; 4099 x 777 float16,
// between words, 13 and 12.
template <typename T, Move MOVE, int TPR, int RUNS>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_sandwich_fwd(const __grid_constant__ SandwichFwdArgs a) {
    RS_PDL_ENTER();
    constexpr bool VEC = MOVE != kAny, FULL = MOVE == kFull;
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1, kKept = power_of_two(3 * RUNS), kForms = power_of_two(RUNS);
    __shared__ float smem[2][16];
    const int t = threadIdx.x % TPR, of = t & 15;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool in = row < a.rows;
    if (TPR == 32 && !in) return;            // a warp without a row; no barrier waits for it
    const long long at = in ? row : 0;
    const T* x = static_cast<const T*>(a.x.p) + at * a.x.stride;
    const T* r = static_cast<const T*>(a.r.p) + at * a.r.stride;
    const T* z = a.gate ? static_cast<const T*>(a.z.p) + at * a.z.stride : nullptr;
    const auto column = [&](int i) { return (i * TPR + t) * 8; };
    // Of a run: how many of its values exist.  Widths are given to threads so that only the last runs may lack some (with
    // four, the last two); threads without a row take the first one's, and store nothing.
    const auto whole = [&](int i) { return FULL || (RUNS < 4 && i + 1 < RUNS); };
    const auto rest = [&](int i) {
        return whole(i) ? 8 : !in ? 0 : MOVE == kRuns ? (column(i) < a.cols ? 8 : 0) : a.cols - column(i);
    };
    Run8<T> xv[RUNS], rv[RUNS], zv[RUNS];
    const auto load = [&](Run8<T>& v, const T* p, int i) {
        if constexpr (VEC) v.template load<true>(p + column(i), rest(i));
        else v.load_words(p + column(i), rest(i));
    };
#pragma unroll
    for (int i = 0; i < RUNS; ++i) load(rv[i], r, i);
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        load(xv[i], x, i);
        if (a.gate == kElementGate) load(zv[i], z, i);
    }
    const float row_gate = a.gate == kRowGate ? gate_of(gate_e(to_f(z[0]))) : 1.f;
    float2 ss = f2(0.f);
#pragma unroll
    for (int i = 0; i < RUNS; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p) ss = f2_fma(rv[i].pair(p), rv[i].pair(p), ss);
    float sums[1] = {ss.x + ss.y};
    row_sums<TPR>(sums, smem[0]);
    const float rstd_r = 1.0f / sqrtf(sums[0] * a.inv_cols + a.eps);
    if (in && t == 0 && a.rstd_r) a.rstd_r[row] = rstd_r;

    // The operands' 8-bit forms: value 3 i + k is run i's operand k.
    if (a.kx.q || a.kr.q || a.kz.q) {
        float m[kKept], scale, inv;
#pragma unroll
        for (int i = 0; i < kKept; ++i) m[i] = 0.f;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            m[3 * i] = max_abs8(xv[i]);
            m[3 * i + 1] = max_abs8(rv[i]);
            // gates beyond that become the largest 8-bit value
            if (a.kz.q) m[3 * i + 2] = fminf(max_abs8(zv[i]), kGateEnd);
        }
        max_over_16(m, of);
        block_scale(m[0], scale, inv);
        const auto keep = [&](const Form& f, const Run8<T> (&v)[RUNS], int k) {
            if (!f.q) return;
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                constexpr int kEach = 16 / kKept;
                const int c = column(i), first = (3 * i + k) * kEach;
                const float by = __shfl_sync(0xffffffffu, inv, first, 16);
                if (of == first && in && (whole(i) || c - of * 8 < a.cols))
                    f.scales[size_t(c / kBlock) * a.rows + row] = scale;
                const float2 w[4] = {v[i].pair(0), v[i].pair(1), v[i].pair(2), v[i].pair(3)};
                if (in && rest(i) > 0) store_e4m3(f.q + row * f.stride + c, rest(i), w, by);
            }
        };
        keep(a.kx, xv, 0);
        keep(a.kr, rv, 1);
        keep(a.kz, zv, 2);
    }

    float2 v[RUNS][4];
    ss = f2(0.f);
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        float2 g[4], w[4];
        if (a.gate == kElementGate) {
#pragma unroll
            for (int p = 0; p < 4; ++p) g[p] = gate_of(gate_e(zv[i].pair(p)));
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) g[p] = f2(row_gate);
        }
        load_vector<VEC>(a.wpost + column(i), rest(i), a.wide, w);
#pragma unroll
        for (int p = 0; p < 4; ++p) g[p] = f2_mul(g[p], f2_mul(f2_mul(rv[i].pair(p), f2(rstd_r)), w[p]));
        if (a.alpha) {
            load_vector<VEC>(a.alpha + column(i), rest(i), a.wide, w);
#pragma unroll
            for (int p = 0; p < 4; ++p) v[i][p] = f2_fma(w[p], xv[i].pair(p), g[p]);
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) v[i][p] = f2_fma(f2(1.f), xv[i].pair(p), g[p]);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) ss = f2_fma(v[i][p], v[i][p], ss);
    }
    sums[0] = ss.x + ss.y;
    row_sums<TPR>(sums, smem[1]);
    const float rstd_s = 1.0f / sqrtf(sums[0] * a.inv_cols + a.eps);
    if (in && t == 0 && a.rstd_s) a.rstd_s[row] = rstd_s;
    if (a.sum && in) {
#pragma unroll
        for (int i = 0; i < RUNS; ++i)
            store_pairs<T, VEC>(static_cast<T*>(a.sum) + row * a.sums + column(i), rest(i), v[i]);
    }
    float top[kForms];
#pragma unroll
    for (int i = 0; i < kForms; ++i) top[i] = 0.f;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        float2 w[4];
        load_vector<VEC>(a.wpre + column(i), rest(i), a.wide, w);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            v[i][p] = f2_mul(f2_mul(v[i][p], f2(rstd_s)), w[p]);
            top[i] = fmaxf(top[i], fmaxf(fabsf(v[i][p].x), fabsf(v[i][p].y)));
        }
        if (a.y && in && rest(i) > 0)
            store_pairs<T, VEC>(static_cast<T*>(a.y) + row * a.ys + column(i), rest(i), v[i]);
    }
    if (!a.q.q) return;
    float scale, inv;
    max_over_16(top, of);
    block_scale(top[0], scale, inv);
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        constexpr int kEach = 16 / kForms;
        const int c = column(i);
        const float by = __shfl_sync(0xffffffffu, inv, i * kEach, 16);
        if (of == i * kEach && in && (whole(i) || c - of * 8 < a.cols)) a.q.scales[size_t(c / kBlock) * a.rows + row] = scale;
        if (in && rest(i) > 0) store_e4m3(a.q.q + row * a.q.stride + c, rest(i), v[i], by);
    }
}

template <typename T, Move MOVE, int TPR, int RUNS>
cudaError_t fwd(const SandwichFwdArgs& a, cudaStream_t s) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    return pdl_launch(k_sandwich_fwd<T, MOVE, TPR, RUNS>, ceil_div(a.rows, kRows), TPR < 128 ? 128 : TPR, 0, s, a);
}

template <typename T, int TPR, int RUNS>
cudaError_t fwd_moved(const SandwichFwdArgs& a, bool vec, cudaStream_t s) {
    if (!vec) return fwd<T, kAny, TPR, RUNS>(a, s);
    return a.cols == 8 * TPR * RUNS ? fwd<T, kFull, TPR, RUNS>(a, s) : fwd<T, kRuns, TPR, RUNS>(a, s);
}

// Two or three runs a thread from 129 columns on, on as few threads as they fit (512 columns on 64 threads with one run
// each: 384 against 243 us, with the arithmetic one by one; 100,000 x 768 bf16 on 32 threads with three 151 us, on 64 with
// two, of which a quarter are idle, 217).  125,000 x 640 192 us, 223 where every run asked whether it exists; kFull, where
// none does: 250,000 x 512 243 us, 273 as kRuns.
template <typename T>
cudaError_t fwd_width(const SandwichFwdArgs& a, bool vec, cudaStream_t s) {
    const int runs = ceil_div(a.cols, 8);
    if (runs <= 16) return fwd_moved<T, 16, 1>(a, vec, s);
    if (runs <= 32) return fwd_moved<T, 16, 2>(a, vec, s);
    if (runs <= 48) return fwd_moved<T, 16, 3>(a, vec, s);
    if (runs <= 64) return fwd_moved<T, 32, 2>(a, vec, s);
    if (runs <= 96) return fwd_moved<T, 32, 3>(a, vec, s);
    if (runs <= 128) return fwd_moved<T, 64, 2>(a, vec, s);
    if (runs <= 192) return fwd_moved<T, 64, 3>(a, vec, s);
    if (runs <= 256) return fwd_moved<T, 128, 2>(a, vec, s);
    if (runs <= 384) return fwd_moved<T, 128, 3>(a, vec, s);
    if (runs <= 512) return fwd_moved<T, 256, 2>(a, vec, s);
    if (runs <= 768) return fwd_moved<T, 256, 3>(a, vec, s);
    if (runs <= 1024) return fwd_moved<T, 512, 2>(a, vec, s);
    return fwd_moved<T, 512, 4>(a, vec, s);
}

}  // namespace
}  // namespace rs

extern "C" {

int rs_sandwich_norm_fwd(const rs_sandwich* block, float eps, const rs_sandwich_out* out, void* stream) {
    using namespace rs;
    if (!block || !out || !(eps >= 0.f) || !isfinite(eps)) return RS_ERR_INVALID_ARG;
    bool kept, vec;
    if (!operands_ok(block, kept, vec) || kept) return RS_ERR_INVALID_ARG;
    if (block->rows == 0) return RS_OK;
    const int32_t cols = block->cols, dtype = block->dtype;
    const size_t z = dtype_size(dtype);
    if (out->d_sum) {
        if (!matrix_ok(out->d_sum, out->sum_stride, cols, dtype)) return RS_ERR_INVALID_ARG;
        if ((out->d_sum == block->d_x && out->sum_stride != block->x_stride) ||
            (out->d_sum == block->d_r && out->sum_stride != block->r_stride))
            return RS_ERR_INVALID_ARG;
        vec = vec && rows16(out->d_sum, out->sum_stride, z);
    }
    if (out->d_y) {
        if (!matrix_ok(out->d_y, out->y_stride, cols, dtype)) return RS_ERR_INVALID_ARG;
        vec = vec && rows16(out->d_y, out->y_stride, z);
    }
    if (!out->q.d_q && !out->d_y) return RS_ERR_INVALID_ARG;
    for (const rs_fp8_matrix* f : {&out->q, &out->kept_x, &out->kept_r, &out->kept_gate})
        if (!form_ok(*f, cols)) return RS_ERR_INVALID_ARG;
    if (out->kept_gate.d_q && block->gate_cols <= 1) return RS_ERR_INVALID_ARG;
    if ((out->d_rstd_r && !ptr_ok(out->d_rstd_r, 4)) || (out->d_rstd_s && !ptr_ok(out->d_rstd_s, 4)))
        return RS_ERR_INVALID_ARG;
    const auto form = [](const rs_fp8_matrix& f) { return Form{f.d_q, f.stride, f.d_scales}; };
    const SandwichFwdArgs a{args_of(block), eps, out->d_sum, out->sum_stride, out->d_y, out->y_stride, form(out->q),
                            form(out->kept_x), form(out->kept_r), form(out->kept_gate), out->d_rstd_r, out->d_rstd_s};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        return fwd_width<T>(a, vec, s);
    });
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
