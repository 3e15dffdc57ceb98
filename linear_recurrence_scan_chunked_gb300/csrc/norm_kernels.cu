// norm_kernels.cu -- layer norm over the last axis of [N, D], forward (with
// the residual add fused) and backward (with the reductions of the weight's
// and the bias's gradients).
//
// Forward, per row:  s = x + res (rounded to the storage type: it is an output,
//   and the norm is taken of what is kept),  mean = sum s / D,
//   var = sum (s - mean)^2 / D,  rstd = 1 / sqrt(var + eps),
//   y = (s - mean) rstd w + b.
// Backward, per row:  xh = (s - mean) rstd,  t = dy w,
//   dx = rstd (t - mean(t) - xh mean(t xh)) + dres,
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// Every element crosses HBM once: a row lives in the registers of T threads
// (NV vectors each), so the mean, the squared deviations from it (two passes
// over registers: no cancellation) and the output need no second read.  CTAs
// are persistent over the rows, which keeps w and b, and backward the columns'
// partial sums, in registers; backward each CTA leaves one row of partial sums
// and a second kernel adds them in a fixed order (bitwise reproducible).
#include "lr_launch.h"

namespace lrs {

// Sum of `v` over the T = 32*W threads of a row (blockDim.x), to all of them.
// sm: [blockDim.y][32] floats; two buffers alternate so that one barrier per
// reduction is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* sm) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    const int W = blockDim.x >> 5;
    if (W == 1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* row = sm + threadIdx.y * (32 * N);
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) row[k * 32 + warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float t = lane < W ? row[k * 32 + lane] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        v[k] = t;
    }
}

template <typename S, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_ln_fwd(const S* __restrict__ x, const S* __restrict__ res, const float* __restrict__ w,
             const float* __restrict__ b, S* __restrict__ y, S* __restrict__ sum,
             float* __restrict__ mean, float* __restrict__ rstd, int64_t N, int D, float eps) {
    __shared__ float sm[2][8][32];  // at most 8 rows a CTA (256 threads of 32)
    const int T = blockDim.x;
    const float inv_d = 1.f / (float)D;
    bool in[NV];
    float wv[NV][VEC], bv[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int d = (k * T + (int)threadIdx.x) * VEC;
        in[k] = d < D;
#pragma unroll
        for (int v = 0; v < VEC; ++v) { wv[k][v] = 0.f; bv[k][v] = 0.f; }
        if (in[k]) {
            load_param<VEC>(w + d, wv[k]);
            if (b != nullptr) load_param<VEC>(b + d, bv[k]);
        }
    }
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    // every row of a CTA runs the same number of rounds (the barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < N; r0 += step) {
        const int64_t r = r0 + threadIdx.y;
        const bool live = r < N;
        const int64_t base = r * D;
        float e[NV][VEC];
        float t[1] = {0.f};
        Pack<S, VEC> px[NV], pr[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * T + (int)threadIdx.x) * VEC;
            px[k].ident(0.f);
            pr[k].ident(0.f);
            if (live && in[k]) {
                px[k].load(x + base + d);
                if (res != nullptr) pr[k].load(res + base + d);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * T + (int)threadIdx.x) * VEC;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                e[k][v] = px[k].get(v);
                if (res != nullptr) {
                    e[k][v] += pr[k].get(v);
                    if constexpr (sizeof(S) == 2) e[k][v] = bf_lo(bf_bits(e[k][v]));
                }
                t[0] += e[k][v];
            }
            if (res != nullptr && live && in[k]) store_vec<S, VEC>(sum + base + d, e[k]);
        }
        row_sum(t, &sm[0][0][0]);
        const float mu = t[0] * inv_d;
        t[0] = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float c = in[k] ? e[k][v] - mu : 0.f;
                t[0] = fmaf(c, c, t[0]);
            }
        row_sum(t, &sm[1][0][0]);
        const float rs = 1.f / sqrtf(fmaf(t[0], inv_d, eps));
        if (live) {
            if (threadIdx.x == 0) {
                mean[r] = mu;
                rstd[r] = rs;
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int d = (k * T + (int)threadIdx.x) * VEC;
                float o[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[v] = fmaf((e[k][v] - mu) * rs, wv[k][v], bv[k][v]);
                if (in[k]) store_vec<S, VEC>(y + base + d, o);
            }
        }
    }
}

// partials: [2][gridDim.x][D] (dw, db).
template <typename S, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_ln_bwd(const S* __restrict__ x, const float* __restrict__ w, const float* __restrict__ mean,
             const float* __restrict__ rstd, const S* __restrict__ dy, const S* __restrict__ dres,
             S* __restrict__ dx, float* __restrict__ partials, int64_t N, int D) {
    __shared__ float sm[2][8][64];
    extern __shared__ float cols[];  // [blockDim.y - 1][T * NV * VEC] when a CTA holds several rows
    const int T = blockDim.x;
    const float inv_d = 1.f / (float)D;
    bool in[NV];
    float wv[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int d = (k * T + (int)threadIdx.x) * VEC;
        in[k] = d < D;
#pragma unroll
        for (int v = 0; v < VEC; ++v) wv[k][v] = aw[k][v] = ab[k][v] = 0.f;
        if (in[k]) load_param<VEC>(w + d, wv[k]);
    }
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int par = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < N; r0 += step, par ^= 1) {
        const int64_t r = r0 + threadIdx.y;
        const bool live = r < N;
        const int64_t base = r * D;
        Pack<S, VEC> px[NV], pd[NV], pr[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * T + (int)threadIdx.x) * VEC;
            px[k].ident(0.f);
            pd[k].ident(0.f);
            pr[k].ident(0.f);
            if (live && in[k]) {
                px[k].load(x + base + d);
                pd[k].load(dy + base + d);
                if (dres != nullptr) pr[k].load(dres + base + d);
            }
        }
        const float mu = live ? __ldg(mean + r) : 0.f, rs = live ? __ldg(rstd + r) : 0.f;
        float t[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float xh = in[k] ? (px[k].get(v) - mu) * rs : 0.f;
                const float g = pd[k].get(v);
                aw[k][v] = fmaf(g, xh, aw[k][v]);
                ab[k][v] += g;
                const float q = g * wv[k][v];
                t[0] += q;
                t[1] = fmaf(q, xh, t[1]);
            }
        row_sum(t, &sm[par][0][0]);
        const float c0 = t[0] * inv_d, c1 = t[1] * inv_d;
        if (live) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int d = (k * T + (int)threadIdx.x) * VEC;
                float o[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float xh = (px[k].get(v) - mu) * rs;
                    o[v] = fmaf(rs, pd[k].get(v) * wv[k][v] - c0 - xh * c1, pr[k].get(v));
                }
                if (in[k]) store_vec<S, VEC>(dx + base + d, o);
            }
        }
    }
    // the CTA's rows of columns: row 0 adds the others' in order
    const int pitch = T * NV * VEC;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        if (blockDim.y > 1) {
            __syncthreads();
            if (threadIdx.y > 0) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        cols[(threadIdx.y - 1) * pitch + (k * VEC + v) * T + threadIdx.x] = a == 0 ? aw[k][v] : ab[k][v];
            }
            __syncthreads();
        }
        if (threadIdx.y == 0) {
            float* out = partials + ((int64_t)a * gridDim.x + blockIdx.x) * D;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int d = (k * T + (int)threadIdx.x) * VEC;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float s = a == 0 ? aw[k][v] : ab[k][v];
                    for (int j = 0; j + 1 < (int)blockDim.y; ++j) s += cols[j * pitch + (k * VEC + v) * T + threadIdx.x];
                    if (in[k]) out[d + v] = s;
                }
            }
        }
    }
}

// dw and db: the G partial rows of each, added in a fixed order.  A block owns
// 32 columns (x) of one of the two arrays; its 32 lanes (y) sum every 32nd row.
__global__ void __launch_bounds__(1024)
    k_ln_colsum(const float* __restrict__ partials, int G, int64_t D, float* __restrict__ dw,
                float* __restrict__ db) {
    __shared__ float part[32][33];
    const int64_t d = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const float* p = partials + (int64_t)blockIdx.y * G * D + d;
    float acc = 0.f;
    if (d < D)
        for (int k = threadIdx.y; k < G; k += 32) acc += __ldg(p + (int64_t)k * D);
    part[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    // transposed: warp j sums column j's 32 lanes
    float s = part[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const int64_t dj = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && dj < D) (blockIdx.y == 0 ? dw : db)[dj] = s;
}

// Threads of a row and vectors of a thread: the fewest vectors that keep a row
// within 256 threads, up to 16 elements a thread (rows short of 256 threads
// share a CTA); wider rows take up to 512 threads, and past 16 x 512 elements
// 32 a thread.
struct LnShape {
    int nv, t, rows;
};
static LnShape ln_shape(int64_t D, int vec) {
    LnShape s{1, 0, 1};
    auto lanes = [&](int nv) { return (D + (int64_t)vec * nv - 1) / ((int64_t)vec * nv); };
    while (vec * s.nv < 16 && lanes(s.nv) > 256) s.nv *= 2;
    if (lanes(s.nv) > 512) s.nv *= 2;
    s.t = (int)((lanes(s.nv) + 31) / 32 * 32);
    s.rows = s.t >= 256 ? 1 : 256 / s.t;
    return s;
}

template <class K>
static int ln_grid(K kernel, int threads, size_t smem, int64_t groups) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n <= 0) n = 1;
    const int64_t cap = (int64_t)n * sm_count();
    return (int)(groups < cap ? groups : cap);
}

template <typename S, int VEC, int NV, int MAXT>
static cudaError_t ln_fwd_k(const LnShape& sh, const void* x, const void* res, const float* w,
                            const float* b, void* y, void* sum, float* mean, float* rstd, int64_t N,
                            int64_t D, float eps, cudaStream_t s) {
    const int grid = ln_grid(k_ln_fwd<S, VEC, NV, MAXT>, sh.t * sh.rows, 0, (N + sh.rows - 1) / sh.rows);
    k_ln_fwd<S, VEC, NV, MAXT><<<grid, dim3(sh.t, sh.rows), 0, s>>>(
        (const S*)x, (const S*)res, w, b, (S*)y, (S*)sum, mean, rstd, N, (int)D, eps);
    return cudaGetLastError();
}

template <typename S, int VEC, int NV, int MAXT>
static cudaError_t ln_bwd_k(const LnShape& sh, const void* x, const float* w, const float* mean,
                            const float* rstd, const void* dy, const void* dres, void* dx, float* dw,
                            float* db, float* partials, int64_t N, int64_t D, cudaStream_t s) {
    const size_t smem = (size_t)(sh.rows - 1) * sh.t * NV * VEC * sizeof(float);
    int grid = ln_grid(k_ln_bwd<S, VEC, NV, MAXT>, sh.t * sh.rows, smem, (N + sh.rows - 1) / sh.rows);
    if (grid > kLnMaxPartials) grid = kLnMaxPartials;
    k_ln_bwd<S, VEC, NV, MAXT><<<grid, dim3(sh.t, sh.rows), smem, s>>>(
        (const S*)x, w, mean, rstd, (const S*)dy, (const S*)dres, (S*)dx, partials, N, (int)D);
    k_ln_colsum<<<dim3((unsigned)((D + 31) / 32), 2), dim3(32, 32), 0, s>>>(partials, grid, D, dw, db);
    return cudaGetLastError();
}

// The instance of a shape.
#define LN_PICK(CALL)                                                     \
    if (sh.nv == 1) return CALL(1, 256);                                  \
    if constexpr (VEC < 8) {                                              \
        if (sh.nv == 2) return CALL(2, 256);                              \
    }                                                                     \
    if constexpr (VEC < 4) {                                              \
        if (sh.nv == 4) return CALL(4, 256);                              \
        if (sh.nv == 8) return CALL(8, 256);                              \
    }                                                                     \
    if (sh.nv * VEC == 16) return sh.t <= 256 ? CALL((16 / VEC), 256) : CALL((16 / VEC), 512); \
    if (sh.nv * VEC == 32) return CALL((32 / VEC), 512);                  \
    return cudaErrorInvalidValue;

template <typename S, int VEC>
static cudaError_t ln_fwd_t(const void* x, const void* res, const float* w, const float* b, void* y,
                            void* sum, float* mean, float* rstd, int64_t N, int64_t D, float eps,
                            cudaStream_t s) {
    const LnShape sh = ln_shape(D, VEC);
#define CALL(NV, MAXT) ln_fwd_k<S, VEC, NV, MAXT>(sh, x, res, w, b, y, sum, mean, rstd, N, D, eps, s)
    LN_PICK(CALL)
#undef CALL
}
template <typename S, int VEC>
static cudaError_t ln_bwd_t(const void* x, const float* w, const float* mean, const float* rstd,
                            const void* dy, const void* dres, void* dx, float* dw, float* db,
                            float* partials, int64_t N, int64_t D, cudaStream_t s) {
    const LnShape sh = ln_shape(D, VEC);
#define CALL(NV, MAXT) ln_bwd_k<S, VEC, NV, MAXT>(sh, x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s)
    LN_PICK(CALL)
#undef CALL
}

// vec: every pointer 16-byte aligned and D a multiple of the 16-byte vector
cudaError_t launch_ln_fwd(int dtype, bool vec, const void* x, const void* res, const float* w,
                          const float* b, void* y, void* sum, float* mean, float* rstd, int64_t N,
                          int64_t D, float eps, cudaStream_t s) {
    if (dtype == 0)
        return vec ? ln_fwd_t<float, 4>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s)
                   : ln_fwd_t<float, 1>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s);
    return vec ? ln_fwd_t<__nv_bfloat16, 8>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s)
               : ln_fwd_t<__nv_bfloat16, 1>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s);
}

cudaError_t launch_ln_bwd(int dtype, bool vec, const void* x, const float* w, const float* mean,
                          const float* rstd, const void* dy, const void* dres, void* dx, float* dw,
                          float* db, float* partials, int64_t N, int64_t D, cudaStream_t s) {
    if (dtype == 0)
        return vec ? ln_bwd_t<float, 4>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s)
                   : ln_bwd_t<float, 1>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s);
    return vec ? ln_bwd_t<__nv_bfloat16, 8>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s)
               : ln_bwd_t<__nv_bfloat16, 1>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s);
}

}  // namespace lrs
