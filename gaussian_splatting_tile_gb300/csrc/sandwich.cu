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
// gates below 1.8e-35 count as that.
__device__ __forceinline__ float gate_e(float z) {
    const float u = -z;
    return __expf(u > 80.f ? 80.f : u);
}
__device__ __forceinline__ float gate_of(float e) { return __fdividef(1.f, 1.f + e); }

// Sums over the TPR threads of a row.  All threads of the block call it (TPR > 32 uses barriers).
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* smem) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = group_sum<(TPR < 32 ? TPR : 32)>(v[k]);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) smem[(threadIdx.x >> 5) * N + k] = v[k];
        __syncthreads();
        const float* mine = smem + threadIdx.x / TPR * kWarps * N;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) v[k] += mine[i * N + k];
        }
    }
}

// ---------------------------------------------------------------- forward
// A row stays in registers between its sums, as in the plain norm: TPR threads, RUNS runs of eight values each.
template <typename T, bool VEC, int TPR, int RUNS>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_sandwich_fwd(const __grid_constant__ SandwichFwdArgs a) {
    RS_PDL_ENTER();
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    __shared__ float smem[32];
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool in = row < a.rows;
    const long long at = in ? row : 0;
    const T* x = static_cast<const T*>(a.x.p) + at * a.x.stride;
    const T* r = static_cast<const T*>(a.r.p) + at * a.r.stride;
    const T* z = a.gate ? static_cast<const T*>(a.z.p) + at * a.z.stride : nullptr;
    Run8<T> xv[RUNS], rv[RUNS], zv[RUNS];
    float sums[1] = {0.f};
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int c = (i * TPR + t) * 8, left = in ? a.cols - c : 0;
        rv[i].template load<VEC>(r + c, left, c > 0);
        xv[i].template load<VEC>(x + c, left, c > 0);
        if (a.gate == kElementGate) zv[i].template load<VEC>(z + c, left, c > 0);
    }
    const float row_gate = a.gate == kRowGate ? gate_of(gate_e(to_f(z[0]))) : 1.f;
#pragma unroll
    for (int i = 0; i < RUNS; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float2 f = rv[i].pair(p);
            sums[0] = fmaf(f.x, f.x, sums[0]);
            sums[0] = fmaf(f.y, f.y, sums[0]);
        }
    row_sums<TPR>(sums, smem);
    const float rstd_r = 1.0f / sqrtf(sums[0] * a.inv_cols + a.eps);
    if (in && t == 0 && a.rstd_r) a.rstd_r[row] = rstd_r;

    // The operands' 8-bit forms.  Thread 3 i + k of the sixteen that share a block's columns forms the two quotients of
    // run i's operand k, and passes them on.
    const int of = t & 15;
    if (a.kx.q || a.kr.q || a.kz.q) {
        float mine = 0.f, scale, inv;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const float mx = group_max<16>(max_abs8(xv[i])), mr = group_max<16>(max_abs8(rv[i]));
            mine = of == 3 * i ? mx : of == 3 * i + 1 ? mr : mine;
            if (a.kz.q) {
                const float mz = group_max<16>(max_abs8(zv[i]));
                mine = of == 3 * i + 2 ? mz : mine;
            }
        }
        block_scale(mine, scale, inv);
        const auto keep = [&](const Form& f, const Run8<T> (&v)[RUNS], int k) {
            if (!f.q) return;
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                const int c = (i * TPR + t) * 8, left = a.cols - c;
                const float by = __shfl_sync(0xffffffffu, inv, 3 * i + k, 16);
                if (of == 3 * i + k && in && c - of * 8 < a.cols) f.scales[size_t(c / kBlock) * a.rows + row] = scale;
                if (in && left > 0) store8_e4m3(f.q + row * f.stride + c, left, v[i], by);
            }
        };
        keep(a.kx, xv, 0);
        keep(a.kr, rv, 1);
        keep(a.kz, zv, 2);
    }

    float v[RUNS][8];
    sums[0] = 0.f;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int c = (i * TPR + t) * 8, left = in ? a.cols - c : 0;
        float wp[8], al[8];
        load8<float, VEC>(a.wpost + c, left, wp);
        if (a.alpha) load8<float, VEC>(a.alpha + c, left, al);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float2 xx = xv[i].pair(p), rr = rv[i].pair(p);
            float2 g = make_float2(row_gate, row_gate);
            if (a.gate == kElementGate) {
                const float2 zz = zv[i].pair(p);
                g = make_float2(gate_of(gate_e(zz.x)), gate_of(gate_e(zz.y)));
            }
            const float n0 = rr.x * rstd_r * wp[2 * p], n1 = rr.y * rstd_r * wp[2 * p + 1];
            v[i][2 * p] = fmaf(g.x, n0, a.alpha ? xx.x * al[2 * p] : xx.x);
            v[i][2 * p + 1] = fmaf(g.y, n1, a.alpha ? xx.y * al[2 * p + 1] : xx.y);
            sums[0] = fmaf(v[i][2 * p], v[i][2 * p], sums[0]);
            sums[0] = fmaf(v[i][2 * p + 1], v[i][2 * p + 1], sums[0]);
        }
    }
    row_sums<TPR>(sums, smem);
    const float rstd_s = 1.0f / sqrtf(sums[0] * a.inv_cols + a.eps);
    if (in && t == 0 && a.rstd_s) a.rstd_s[row] = rstd_s;
    if (a.sum && in) {
        T* s = static_cast<T*>(a.sum) + row * a.sums;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int c = (i * TPR + t) * 8;
            store8<T, VEC>(s + c, a.cols - c, v[i]);
        }
    }
    float top[RUNS];
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int c = (i * TPR + t) * 8, left = in ? a.cols - c : 0;
        float w[8];
        load8<float, VEC>(a.wpre + c, left, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd_s * w[j];
        if (a.y && left > 0) store8<T, VEC>(static_cast<T*>(a.y) + row * a.ys + c, left, v[i]);
        top[i] = group_max<16>(max_abs8(v[i], 0.f));
    }
    if (!a.q.q) return;
    float mine = top[0], scale, inv;
#pragma unroll
    for (int i = 1; i < RUNS; ++i) mine = of == i ? top[i] : mine;
    block_scale(mine, scale, inv);
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int c = (i * TPR + t) * 8, left = a.cols - c;
        const float by = __shfl_sync(0xffffffffu, inv, i, 16);
        if (of == i && in && c - of * 8 < a.cols) a.q.scales[size_t(c / kBlock) * a.rows + row] = scale;
        if (in && left > 0) store8_e4m3(a.q.q + row * a.q.stride + c, left, v[i], by);
    }
}

template <typename T, bool VEC, int TPR, int RUNS>
cudaError_t fwd(const SandwichFwdArgs& a, cudaStream_t s) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    return pdl_launch(k_sandwich_fwd<T, VEC, TPR, RUNS>, ceil_div(a.rows, kRows), TPR < 128 ? 128 : TPR, 0, s, a);
}

template <typename T, bool VEC>
cudaError_t fwd_width(const SandwichFwdArgs& a, cudaStream_t s) {
    const int runs = ceil_div(a.cols, 8);
    if (runs <= 16) return fwd<T, VEC, 16, 1>(a, s);
    if (runs <= 32) return fwd<T, VEC, 32, 1>(a, s);
    if (runs <= 64) return fwd<T, VEC, 64, 1>(a, s);
    if (runs <= 128) return fwd<T, VEC, 128, 1>(a, s);
    if (runs <= 256) return fwd<T, VEC, 256, 1>(a, s);
    if (runs <= 512) return fwd<T, VEC, 512, 1>(a, s);
    if (runs <= 1024) return fwd<T, VEC, 512, 2>(a, s);
    return fwd<T, VEC, 512, 4>(a, s);
}

// ---------------------------------------------------------------- backward
// Eight values of an operand as they are stored, or of its checkpoint.
template <typename T, bool KEPT, bool VEC>
struct Operand8 {
    Run8<T> v;
    __device__ __forceinline__ void load(const Stored& s, long long row, int, int c, int left) {
        v.template load<VEC>(static_cast<const T*>(s.p) + row * s.stride + c, left, c > 0);
    }
    __device__ __forceinline__ float2 pair(int p) const { return v.pair(p); }
};
template <typename T, bool VEC>
struct Operand8<T, true, VEC> {
    Bytes8 v;
    float scale;
    __device__ __forceinline__ void load(const Stored& s, long long row, int rows, int c, int left) {
        v.load(static_cast<const uint8_t*>(s.p) + row * s.stride + c, left);
        scale = left > 0 ? s.scales[size_t(c / kBlock) * rows + row] : 0.f;
    }
    __device__ __forceinline__ float2 pair(int p) const {
        const float2 f = v.pair(p);
        return make_float2(f.x * scale, f.y * scale);
    }
};

// Everything of eight columns that the two passes over a row need.
template <typename T, bool KEPT, bool VEC>
struct BwdRun {
    Operand8<T, KEPT, VEC> x, r, z;
    Run8<T> dy, ds;
    __device__ __forceinline__ void load(const SandwichBwdArgs& a, long long row, int c, int left) {
        x.load(a.x, row, a.rows, c, left);
        r.load(a.r, row, a.rows, c, left);
        if (a.gate == kElementGate) z.load(a.z, row, a.rows, c, left);
        dy.template load<VEC>(static_cast<const T*>(a.dy) + row * a.dys + c, left, c > 0);
        if (a.ds) ds.template load<VEC>(static_cast<const T*>(a.ds) + row * a.dss + c, left, c > 0);
    }
};
struct BwdRow {
    float rstd_r, rstd_s, e, g;       // e, g: of the row's gate (0, 1 without a gate)
};
struct BwdWeights { float post[8], pre[8], alpha[8]; };

struct BwdValue { float x, rh, n, p, sh, t, e, g, dy, ds; };

template <typename T, bool KEPT, bool VEC>
__device__ __forceinline__ void values(const SandwichBwdArgs& a, const BwdRun<T, KEPT, VEC>& u, const BwdRow& w,
                                       const BwdWeights& k, int p, BwdValue (&o)[2]) {
    const float2 x = u.x.pair(p), r = u.r.pair(p), dy = u.dy.pair(p);
    const float2 ds = a.ds ? u.ds.pair(p) : make_float2(0.f, 0.f);
    const float2 z = a.gate == kElementGate ? u.z.pair(p) : make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        BwdValue& v = o[j];
        v.x = j ? x.y : x.x;
        v.e = w.e;
        v.g = w.g;
        if (a.gate == kElementGate) {
            v.e = gate_e(j ? z.y : z.x);
            v.g = gate_of(v.e);
        }
        v.rh = (j ? r.y : r.x) * w.rstd_r;
        v.n = v.rh * k.post[2 * p + j];
        v.p = v.g * v.n;
        v.sh = fmaf(v.g, v.n, a.alpha ? v.x * k.alpha[2 * p + j] : v.x) * w.rstd_s;
        v.dy = j ? dy.y : dy.x;
        v.t = v.dy * k.pre[2 * p + j];
        v.ds = j ? ds.y : ds.x;
    }
}

// A block takes every gridDim-th group of rows; a thread keeps the same columns throughout, so its shares of the
// vectors' gradients stay with it and leave once per block, to be added up in a fixed order.  WIDE: a thread's columns
// are too many for its registers; it reads a row twice and keeps its shares in shared memory.
template <typename T, bool KEPT, bool VEC, int TPR, int RUNS, bool WIDE>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_sandwich_bwd(const __grid_constant__ SandwichBwdArgs a) {
    RS_PDL_ENTER();
    constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
    __shared__ float smem[kThreads / 32 * 3];
    extern __shared__ float shares[];        // WIDE: [3][RUNS][8][TPR]; else, with several rows a block, [threads][8]
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float acc[WIDE ? 1 : 3][WIDE ? 1 : RUNS][8];
    const auto share = [&](int k, int i, int j) -> float& {
        if constexpr (WIDE) return shares[((k * RUNS + i) * 8 + j) * TPR + t];
        else return acc[k][i][j];
    };
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < RUNS; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) share(k, i, j) = 0.f;
    for (long long base = (long long)blockIdx.x * kRows; base < a.rows; base += (long long)gridDim.x * kRows) {
        const long long row = base + sub;
        const bool in = row < a.rows;
        const long long at = in ? row : 0;
        BwdRow w{in ? a.rstd_r[at] : 0.f, in ? a.rstd_s[at] : 0.f, 0.f, 1.f};
        if (a.gate == kRowGate) {
            w.e = gate_e(to_f(static_cast<const T*>(a.z.p)[at * a.z.stride]));
            w.g = gate_of(w.e);
        }
        BwdRun<T, KEPT, VEC> u[WIDE ? 1 : RUNS];
        float sums[3] = {0.f, 0.f, 0.f};
        BwdWeights k;
        const auto weights = [&](int c) {    // from L1: registers for them would cost blocks of the SM
            const int left = a.cols - c;
            load8<float, VEC>(a.wpost + c, left, k.post);
            load8<float, VEC>(a.wpre + c, left, k.pre);
            if (a.alpha) load8<float, VEC>(a.alpha + c, left, k.alpha);
        };
        const auto first = [&](int i) {
            const int c = (i * TPR + t) * 8;
            weights(c);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                BwdValue v[2];
                values<T, KEPT, VEC>(a, u[WIDE ? 0 : i], w, k, p, v);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    sums[0] = fmaf(v[j].t, v[j].sh, sums[0]);
                    sums[1] = fmaf(fmaf(w.rstd_s, v[j].t, v[j].ds), v[j].p, sums[1]);
                    sums[2] = fmaf(v[j].sh, v[j].p, sums[2]);
                }
            }
        };
        if constexpr (WIDE) {
#pragma unroll 1
            for (int i = 0; i < RUNS; ++i) {
                const int c = (i * TPR + t) * 8;
                u[0].load(a, at, c, in ? a.cols - c : 0);
                first(i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                const int c = (i * TPR + t) * 8;
                u[i].load(a, at, c, in ? a.cols - c : 0);
            }
#pragma unroll
            for (int i = 0; i < RUNS; ++i) first(i);
        }
        row_sums<TPR>(sums, smem);
        const float c1 = w.rstd_s * (sums[0] * a.inv_cols);
        const float dot = fmaf(-c1, sums[2], sums[1]);           // sum of ds p
        const float c2 = dot * a.inv_cols;
        if (a.gate == kRowGate && a.dz && in && t == 0)
            static_cast<T*>(a.dz)[row * a.dzs] = from_f<T>(dot * (w.e * w.g));
        const auto second = [&](int i) {
            const int c = (i * TPR + t) * 8, left = in ? a.cols - c : 0;
            weights(c);
            float dx[8], dr[8], dz[8];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                BwdValue v[2];
                values<T, KEPT, VEC>(a, u[WIDE ? 0 : i], w, k, p, v);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int e = 2 * p + j;
                    const float ds = fmaf(-c1, v[j].sh, fmaf(w.rstd_s, v[j].t, v[j].ds));
                    const float dn = ds * v[j].g;
                    share(0, i, e) = fmaf(v[j].dy, v[j].sh, share(0, i, e));
                    share(1, i, e) = fmaf(dn, v[j].rh, share(1, i, e));
                    share(2, i, e) = fmaf(ds, v[j].x, share(2, i, e));
                    dx[e] = a.alpha ? ds * k.alpha[e] : ds;
                    dr[e] = w.rstd_r * fmaf(-v[j].rh, c2, dn * k.post[e]);
                    dz[e] = ds * v[j].p * (v[j].e * v[j].g);
                }
            }
            if (left > 0) {
                store8<T, VEC>(static_cast<T*>(a.dx) + row * a.dxs + c, left, dx);
                store8<T, VEC>(static_cast<T*>(a.dr) + row * a.drs + c, left, dr);
                if (a.gate == kElementGate && a.dz) store8<T, VEC>(static_cast<T*>(a.dz) + row * a.dzs + c, left, dz);
            }
        };
        if constexpr (WIDE) {
#pragma unroll 1
            for (int i = 0; i < RUNS; ++i) {
                const int c = (i * TPR + t) * 8;
                u[0].load(a, at, c, in ? a.cols - c : 0);
                second(i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < RUNS; ++i) second(i);
        }
    }
    if (!a.part) return;
    float* part = a.part + size_t(blockIdx.x) * 3 * a.cols;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int c = (i * TPR + t) * 8;
            if constexpr (kRows > 1) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 8; ++j) shares[threadIdx.x * 8 + j] = share(k, i, j);
                __syncthreads();
                if (sub == 0)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        for (int o = 1; o < kRows; ++o) share(k, i, j) += shares[(o * TPR + t) * 8 + j];
            }
            if (sub == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < a.cols) part[size_t(k) * a.cols + c + j] = share(k, i, j);
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

// Threads a row: one run a thread up to 4096 columns, beyond that the wide form on 512 threads.
int bwd_threads(int cols) {
    const int runs = ceil_div(cols, 8);
    for (int t = 16; t < 512; t *= 2)
        if (runs <= t) return t;
    return 512;
}
int bwd_blocks(int rows, int cols) {
    const int t = bwd_threads(cols), rows_a_block = t < 128 ? 128 / t : 1;
    const int per = t <= 128 ? 4 : t == 256 ? 2 : 1;
    return std::max(1, std::min(ceil_div(rows, rows_a_block), kSms * per));
}

template <typename T, bool KEPT, bool VEC, int TPR, int RUNS, bool WIDE>
cudaError_t bwd(const SandwichBwdArgs& a, cudaStream_t s) {
    constexpr int kThreads = TPR < 128 ? 128 : TPR;
    constexpr int smem = WIDE ? 3 * RUNS * 8 * TPR * 4 : kThreads > TPR ? kThreads * 8 * 4 : 0;
    const auto kernel = k_sandwich_bwd<T, KEPT, VEC, TPR, RUNS, WIDE>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    return pdl_launch(kernel, bwd_blocks(a.rows, a.cols), kThreads, smem, s, a);
}

template <typename T, bool KEPT, bool VEC>
cudaError_t bwd_width(const SandwichBwdArgs& a, cudaStream_t s) {
    switch (bwd_threads(a.cols)) {
        case 16: return bwd<T, KEPT, VEC, 16, 1, false>(a, s);
        case 32: return bwd<T, KEPT, VEC, 32, 1, false>(a, s);
        case 64: return bwd<T, KEPT, VEC, 64, 1, false>(a, s);
        case 128: return bwd<T, KEPT, VEC, 128, 1, false>(a, s);
        case 256: return bwd<T, KEPT, VEC, 256, 1, false>(a, s);
    }
    if (a.cols <= 4096) return bwd<T, KEPT, VEC, 512, 1, false>(a, s);
    return a.cols <= 8192 ? bwd<T, KEPT, VEC, 512, 2, true>(a, s) : bwd<T, KEPT, VEC, 512, 4, true>(a, s);
}

// ---------------------------------------------------------------- host side
bool matrix_ok(const void* p, size_t stride, int32_t cols, int32_t dtype) {
    return ptr_ok(p, dtype_size(dtype)) && stride >= size_t(cols);
}
bool form_ok(const rs_fp8_matrix& f, int32_t cols) {
    if (!f.d_q && !f.d_scales) return true;
    return fp8_rows_ok(f.d_q, f.stride, cols) && ptr_ok(f.d_scales, 4);
}

// The block's operands; `kept`: whether they are checkpoints.
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
    vec = ptr_ok(b->d_post_weight, 16) && ptr_ok(b->d_pre_weight, 16) &&
          (!b->d_residual_scale || ptr_ok(b->d_residual_scale, 16));
    if (!kept)
        vec = vec && rows16(b->d_x, b->x_stride, z) && rows16(b->d_r, b->r_stride, z) &&
              (!element || rows16(b->d_gate, b->gate_stride, z));
    return true;
}

SandwichArgs args_of(const rs_sandwich* b) {
    return {b->rows, b->cols, b->gate_cols == 0 ? kNoGate : b->gate_cols == 1 ? kRowGate : kElementGate,
            {b->d_x, b->x_stride, b->d_x_scales}, {b->d_r, b->r_stride, b->d_r_scales},
            {b->d_gate, b->gate_stride, b->d_gate_scales}, b->d_residual_scale, b->d_post_weight, b->d_pre_weight,
            1.0f / float(b->cols)};
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
        return vec ? fwd_width<T, true>(a, s) : fwd_width<T, false>(a, s);
    });
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

size_t rs_sandwich_norm_bwd_workspace_size(int32_t rows, int32_t cols) {
    if (rows < 0 || cols < 1 || cols > RS_NORM_MAX_COLS) return 0;
    return size_t(rs::bwd_blocks(rows, cols)) * 3 * cols * sizeof(float);
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
    const bool element = block->gate_cols > 1;
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
    cudaError_t e = with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        if (kept) return vec ? bwd_width<T, true, true>(a, s) : bwd_width<T, true, false>(a, s);
        return vec ? bwd_width<T, false, true>(a, s) : bwd_width<T, false, false>(a, s);
    });
    if (e == cudaSuccess && any)
        e = pdl_launch(k_sandwich_sums, dim3(ceil_div(cols, 32), 3), 1024, 0, s, static_cast<const float*>(a.part),
                       bwd_blocks(rows, cols), cols, Vectors{{vectors[0], vectors[1], vectors[2]}});
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
