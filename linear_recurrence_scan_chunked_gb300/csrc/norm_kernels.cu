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
//
// Bytes bound it where rows are aligned: bf16 131072 x 4096 with the residual 670 us,
// 6.4 TB/s (copy 6.78).  Odd rows are read an element at a time and issue bounds
// them: fp32 30011 x 1111 backward 79 us, 5.1 TB/s.
#include "lr_launch.h"

#include <atomic>
#include <type_traits>
#include <utility>

namespace lrs {

// Sum of `v` over the threads of a row (blockDim.x: W warps, or 8 or 16 lanes of
// one), to all of them.
// sm: [blockDim.y][32] floats; two buffers alternate so that one barrier per
// reduction is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* sm) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        if (off >= (int)blockDim.x) continue;
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    }
    const int W = blockDim.x >> 5;
    if (W <= 1) return;
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

// A thread's columns: vector k starts at column (k T + threadIdx.x) VEC.  Rows are
// addressed by the CTA's first row, the same for all its threads, plus a 32-bit
// offset that no row changes.  Only the last vectors can lie outside (T is rounded
// up to a warp, NV to an instance); their offset is the row's last vector, whose
// data they read and whose results they drop.
template <typename S, int VEC, int NV>
struct Cols {
    static constexpr int kMasked = NV >= 8 && VEC == 1 ? 2 : 1;
    uint32_t off[NV];  // bytes
    int d[NV];
    bool in_[kMasked];
    __device__ __forceinline__ Cols(int D) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            d[k] = (k * (int)blockDim.x + (int)threadIdx.x) * VEC;
            if (k >= NV - kMasked) {
                in_[k - (NV - kMasked)] = d[k] < D;
                if (d[k] >= D) d[k] = D - VEC;
            }
            off[k] = (uint32_t)((threadIdx.y * D + d[k]) * (int)sizeof(S));
        }
    }
    __device__ __forceinline__ bool in(int k) const {
        return k < NV - kMasked ? true : in_[k < NV - kMasked ? 0 : k - (NV - kMasked)];
    }
    template <typename T>
    __device__ __forceinline__ T* at(T* row, int k) const {
        using B = typename std::conditional<std::is_const<T>::value, const char, char>::type;
        return reinterpret_cast<T*>(reinterpret_cast<B*>(row) + off[k]);
    }
};

// CTAs per SM to compile for (256 threads; a row of up to 512 takes what it
// gets): enough rows in flight to cover the memory's latency.  Left to itself the
// compiler spends 128 registers on five elements a thread, and the backward pass
// of 30011 x 1111 took 10% longer.
constexpr int ln_min_ctas(bool bwd, bool res, int elems, int maxt) {
    return maxt > 256       ? 1
           : elems > 8      ? 2
           : bwd || res     ? (elems <= 2 ? 5 : elems <= 4 ? 4 : elems <= 6 && bwd ? 4 : 3)
           : elems <= 4     ? 6
                            : 4;
}
// Rows past 8192 columns (1024 threads, 64 registers each) keep w and b in L1 and,
// backward, the column sums in shared memory, and load no row ahead.
__host__ __device__ constexpr bool ln_wide(int maxt) { return maxt > 512; }

// The next row's vectors are loaded before the current row's sums: a row's two
// reductions and its output then cover the next one's way from memory.
template <typename S, int VEC, int NV, int MAXT, bool RES>
__global__ void __launch_bounds__(MAXT, ln_min_ctas(false, RES, VEC * NV, MAXT))
    k_ln_fwd(const S* __restrict__ x, const S* __restrict__ res, const float* __restrict__ w,
             const float* __restrict__ b, S* __restrict__ y, S* __restrict__ sum,
             float* __restrict__ mean, float* __restrict__ rstd, int64_t N, int D, float eps) {
    __shared__ float sm[2][8][32];  // at most 8 rows a CTA (256 threads of 32)
    const float inv_d = 1.f / (float)D;
    const Cols<S, VEC, NV> cl(D);
    constexpr bool WIDE = ln_wide(MAXT);
    float wv[NV][VEC], bv[NV][VEC];
    auto params = [&](int k) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) bv[k][v] = 0.f;
        load_param<VEC>(w + cl.d[k], wv[k]);
        if (b != nullptr) load_param<VEC>(b + cl.d[k], bv[k]);
    };
    if constexpr (!WIDE) {
#pragma unroll
        for (int k = 0; k < NV; ++k) params(k);
    }
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    Pack<S, VEC> px[NV], pr[NV];
    auto fetch = [&](int64_t r0) {
        if (r0 + threadIdx.y >= N) return;
        const S *xr = x + r0 * D, *rr = res + r0 * D;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            px[k].load(cl.at(xr, k));
            if constexpr (RES) pr[k].load(cl.at(rr, k));
        }
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) { px[k].ident(0.f); pr[k].ident(0.f); }
    fetch((int64_t)blockIdx.x * blockDim.y);
    // every row of a CTA runs the same number of rounds (the barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < N; r0 += step) {
        const bool live = r0 + threadIdx.y < N;
        S *yr = y + r0 * D, *sr = sum + r0 * D;
        if constexpr (WIDE) {
            if (r0 != (int64_t)blockIdx.x * blockDim.y) fetch(r0);
        }
        float e[NV][VEC];
        float t[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) e[k][v] = px[k].get(v);
            if constexpr (RES) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) e[k][v] += pr[k].get(v);
                if constexpr (sizeof(S) == 2 && VEC > 1) {
                    // rounded once, stored and carried on
#pragma unroll
                    for (int v = 0; v < VEC; v += 2) {
                        px[k].w[v / 2] = bf_pack(e[k][v], e[k][v + 1]);
                        e[k][v] = bf_lo(px[k].w[v / 2]);
                        e[k][v + 1] = bf_hi(px[k].w[v / 2]);
                    }
                    if (live && cl.in(k)) {
                        if constexpr (VEC == 8)
                            st_u4(cl.at(sr, k), make_uint4(px[k].w[0], px[k].w[1], px[k].w[2], px[k].w[3]));
                        else
                            st_u2(cl.at(sr, k), make_uint2(px[k].w[0], px[k].w[1]));
                    }
                } else {
                    if constexpr (sizeof(S) == 2) {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) e[k][v] = bf_lo(bf_bits(e[k][v]));
                    }
                    if (live && cl.in(k)) store_vec<S, VEC>(cl.at(sr, k), e[k]);
                }
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) t[0] += cl.in(k) ? e[k][v] : 0.f;
        }
        if constexpr (!WIDE) fetch(r0 + step);
        row_sum(t, &sm[0][0][0]);
        const float mu = t[0] * inv_d;
        t[0] = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                e[k][v] -= mu;
                const float c = cl.in(k) ? e[k][v] : 0.f;
                t[0] = fmaf(c, c, t[0]);
            }
        row_sum(t, &sm[1][0][0]);
        const float rs = 1.f / sqrtf(fmaf(t[0], inv_d, eps));
        if (live) {
            if (threadIdx.x == 0) {
                mean[r0 + threadIdx.y] = mu;
                rstd[r0 + threadIdx.y] = rs;
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float o[VEC];
                if constexpr (WIDE) params(k);
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[v] = fmaf(e[k][v] * rs, wv[k][v], bv[k][v]);
                if (cl.in(k)) store_vec<S, VEC>(cl.at(yr, k), o);
            }
        }
    }
}

// partials: [2][gridDim.x][D] (dw, db).
template <typename S, int VEC, int NV, int MAXT, bool RES>
__global__ void __launch_bounds__(MAXT, ln_min_ctas(true, RES, VEC * NV, MAXT))
    k_ln_bwd(const S* __restrict__ x, const float* __restrict__ w, const float* __restrict__ mean,
             const float* __restrict__ rstd, const S* __restrict__ dy, const S* __restrict__ dres,
             S* __restrict__ dx, float* __restrict__ partials, int64_t N, int D) {
    __shared__ float sm[2][8][64];
    constexpr bool WIDE = ln_wide(MAXT);
    // several rows a CTA: [blockDim.y - 1][T * NV * VEC] at the end; WIDE: the
    // column sums, [2][NV * VEC][T]
    extern __shared__ float cols[];
    const int T = blockDim.x;
    const float inv_d = 1.f / (float)D;
    const Cols<S, VEC, NV> cl(D);
    float wv[NV][VEC], aw[NV][VEC], ab[NV][VEC];
    auto params = [&](int k) {
        load_param<VEC>(w + cl.d[k], wv[k]);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (!cl.in(k)) wv[k][v] = 0.f;
    };
    auto slot = [&](int a, int k, int v) -> float& { return cols[((a * NV + k) * VEC + v) * T + threadIdx.x]; };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if constexpr (!WIDE) params(k);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if constexpr (WIDE) slot(0, k, v) = slot(1, k, v) = 0.f;
            else aw[k][v] = ab[k][v] = 0.f;
        }
    }
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    Pack<S, VEC> px[NV], pd[NV], pr[NV];
    float mu = 0.f, rs = 0.f;
    auto fetch = [&](int64_t r0) {
        if (r0 + threadIdx.y >= N) {  // past the end: rows of zeros
#pragma unroll
            for (int k = 0; k < NV; ++k) { px[k].ident(0.f); pd[k].ident(0.f); pr[k].ident(0.f); }
            mu = rs = 0.f;
            return;
        }
        const S *xr = x + r0 * D, *gr = dy + r0 * D, *rr = dres + r0 * D;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            px[k].load(cl.at(xr, k));
            pd[k].load(cl.at(gr, k));
            if constexpr (RES) pr[k].load(cl.at(rr, k));
        }
        mu = __ldg(mean + r0 + threadIdx.y);
        rs = __ldg(rstd + r0 + threadIdx.y);
    };
    fetch((int64_t)blockIdx.x * blockDim.y);
    int par = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < N; r0 += step, par ^= 1) {
        const bool live = r0 + threadIdx.y < N;
        S* xr = dx + r0 * D;
        if constexpr (WIDE) {
            if (r0 != (int64_t)blockIdx.x * blockDim.y) fetch(r0);
        }
        // xh, and t = dy w with what dx adds to it: rs t + dres
        float xh[NV][VEC], q[NV][VEC], o[NV][VEC];
        float t[2] = {0.f, 0.f};
        const float r_s = rs;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if constexpr (WIDE) params(k);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                xh[k][v] = (px[k].get(v) - mu) * r_s;
                const float g = pd[k].get(v);
                if constexpr (WIDE) {
                    slot(0, k, v) = fmaf(g, xh[k][v], slot(0, k, v));
                    slot(1, k, v) += g;
                } else {
                    aw[k][v] = fmaf(g, xh[k][v], aw[k][v]);
                    ab[k][v] += g;
                }
                q[k][v] = g * wv[k][v];
                t[0] += q[k][v];
                t[1] = fmaf(q[k][v], xh[k][v], t[1]);
                if constexpr (RES) o[k][v] = pr[k].get(v);
                else o[k][v] = 0.f;
            }
        }
        if constexpr (!WIDE) fetch(r0 + step);
        row_sum(t, &sm[par][0][0]);
        const float c0 = t[0] * inv_d, c1 = t[1] * inv_d;
        if (live) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[k][v] = fmaf(r_s, fmaf(-xh[k][v], c1, q[k][v] - c0), o[k][v]);
                if (cl.in(k)) store_vec<S, VEC>(cl.at(xr, k), o[k]);
            }
        }
    }
    griddep_launch_dependents();
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
                        if constexpr (!WIDE)
                            cols[(threadIdx.y - 1) * pitch + (k * VEC + v) * T + threadIdx.x] = a == 0 ? aw[k][v] : ab[k][v];
            }
            __syncthreads();
        }
        if (threadIdx.y == 0) {
            float* out = partials + ((int64_t)a * gridDim.x + blockIdx.x) * D;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int d = cl.d[k];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float s;
                    if constexpr (WIDE) s = slot(a, k, v);
                    else s = a == 0 ? aw[k][v] : ab[k][v];
                    for (int j = 0; j + 1 < (int)blockDim.y; ++j) s += cols[j * pitch + (k * VEC + v) * T + threadIdx.x];
                    if (cl.in(k)) out[d + v] = s;
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
    griddep_wait();
    if (d < D) {
        int k = threadIdx.y;
        for (; k + 224 < G; k += 256) {  // eight loads in flight, added in order
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = __ldg(p + (int64_t)(k + 32 * u) * D);
#pragma unroll
            for (int u = 0; u < 8; ++u) acc += v[u];
        }
#pragma unroll 4
        for (; k < G; k += 32) acc += __ldg(p + (int64_t)k * D);
    }
    part[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    // transposed: warp j sums column j's 32 lanes
    float s = part[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const int64_t dj = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && dj < D) (blockIdx.y == 0 ? dw : db)[dj] = s;
}

// Threads of a row and vectors of a thread.  Up to 2048 columns about 8 elements a
// thread in 8 to 256 threads -- a warp to one row of up to 256 columns, to two of up
// to 128, to four of up to 64, so that the sums need no barrier; rows short of 256
// threads share a CTA.  (A whole warp for each row of 128 columns, 500000 of them
// in bf16: 88 us forward and 156 backward with dres, where 16 lanes take 51 and
// 100; 647574 rows of 49 backward 127 against 68.)  Up to 4096 columns
// 16 elements (8 one by one, in up to 512 threads), up to 8192 16 in 512 threads,
// beyond 16 in 1024.
struct LnShape {
    int nv, t, rows, maxt;
};
static LnShape ln_shape(int64_t D, int vec) {
    LnShape s{1, 0, 1, 256};
    auto per = [&](int64_t n) { return (D + n - 1) / n; };
    if (D <= 2048) {
        int tm = 8;
        while (tm < 256 && D > 8 * (int64_t)tm) tm *= 2;
        s.nv = (int)per((int64_t)vec * tm);
        if (tm < 32) s.t = tm;
    } else if (D <= 4096) {
        s.nv = vec > 1 ? 16 / vec : 8;
    } else {
        s.nv = 16 / vec;
    }
    if (s.t == 0) s.t = (int)((per((int64_t)vec * s.nv) + 31) / 32 * 32);
    s.maxt = s.t <= 256 ? 256 : s.t <= 512 ? 512 : 1024;
    s.rows = s.t >= 256 ? 1 : 256 / s.t;
    return s;
}

// CTAs of a launch: the groups of rows, at most as many as are resident at once
// (asked once per kernel, device and block size: `known`, one entry per warp count).
// Atomic: the forward call takes no lock, and calls of several threads meet here.
using LnKnown = std::atomic<int>[64][33];
template <class K>
static int ln_grid(K kernel, int threads, size_t smem, int64_t groups, LnKnown& known) {
    int dev = 0;
    cudaGetDevice(&dev);
    std::atomic<int>& slot = known[dev & 63][threads / 32];
    int n = slot.load(std::memory_order_relaxed);
    if (n <= 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n <= 0) n = 1;
        slot.store(n, std::memory_order_relaxed);
    }
    const int64_t cap = (int64_t)n * sm_count();
    return (int)(groups < cap ? groups : cap);
}

template <typename S, int VEC, int NV, int MAXT, bool RES>
static cudaError_t ln_fwd_r(const LnShape& sh, const void* x, const void* res, const float* w,
                            const float* b, void* y, void* sum, float* mean, float* rstd, int64_t N,
                            int64_t D, float eps, cudaStream_t s) {
    static LnKnown known;  // zeros
    const int grid = ln_grid(k_ln_fwd<S, VEC, NV, MAXT, RES>, sh.t * sh.rows, 0, (N + sh.rows - 1) / sh.rows, known);
    k_ln_fwd<S, VEC, NV, MAXT, RES><<<grid, dim3(sh.t, sh.rows), 0, s>>>(
        (const S*)x, (const S*)res, w, b, (S*)y, (S*)sum, mean, rstd, N, (int)D, eps);
    return cudaGetLastError();
}

template <typename S, int VEC, int NV, int MAXT, bool RES>
static cudaError_t ln_bwd_r(const LnShape& sh, const void* x, const float* w, const float* mean,
                            const float* rstd, const void* dy, const void* dres, void* dx, float* dw,
                            float* db, float* partials, int64_t N, int64_t D, cudaStream_t s) {
    const size_t smem = (size_t)(ln_wide(MAXT) ? 2 : sh.rows - 1) * sh.t * NV * VEC * sizeof(float);
    if (ln_wide(MAXT)) {
        const cudaError_t e = cudaFuncSetAttribute(k_ln_bwd<S, VEC, NV, MAXT, RES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   2 * 1024 * 16 * (int)sizeof(float));
        if (e != cudaSuccess) return e;
    }
    static LnKnown known;  // zeros
    int grid = ln_grid(k_ln_bwd<S, VEC, NV, MAXT, RES>, sh.t * sh.rows, smem, (N + sh.rows - 1) / sh.rows, known);
    if (grid > kLnMaxPartials) grid = kLnMaxPartials;
    k_ln_bwd<S, VEC, NV, MAXT, RES><<<grid, dim3(sh.t, sh.rows), smem, s>>>(
        (const S*)x, w, mean, rstd, (const S*)dy, (const S*)dres, (S*)dx, partials, N, (int)D);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_dep(k_ln_colsum, dim3((unsigned)((D + 31) / 32), 2), dim3(32, 32), 0, s, (const float*)partials, grid, D, dw,
                      db);
}

template <typename S, int VEC, int NV, int MAXT>
static cudaError_t ln_fwd_k(const LnShape& sh, const void* x, const void* res, const float* w,
                            const float* b, void* y, void* sum, float* mean, float* rstd, int64_t N,
                            int64_t D, float eps, cudaStream_t s) {
    return res ? ln_fwd_r<S, VEC, NV, MAXT, true>(sh, x, res, w, b, y, sum, mean, rstd, N, D, eps, s)
               : ln_fwd_r<S, VEC, NV, MAXT, false>(sh, x, res, w, b, y, sum, mean, rstd, N, D, eps, s);
}
template <typename S, int VEC, int NV, int MAXT>
static cudaError_t ln_bwd_k(const LnShape& sh, const void* x, const float* w, const float* mean,
                            const float* rstd, const void* dy, const void* dres, void* dx, float* dw,
                            float* db, float* partials, int64_t N, int64_t D, cudaStream_t s) {
    return dres ? ln_bwd_r<S, VEC, NV, MAXT, true>(sh, x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s)
                : ln_bwd_r<S, VEC, NV, MAXT, false>(sh, x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s);
}

// The instance of a shape.
#define LN_PICK(CALL)                                                     \
    if (sh.maxt == 1024) return CALL((16 / VEC), 1024);                   \
    if (sh.maxt == 512) {                                                 \
        if constexpr (VEC == 1) {                                         \
            if (sh.nv == 8) return CALL(8, 512);                          \
        }                                                                 \
        return CALL((16 / VEC), 512);                                     \
    }                                                                     \
    switch (sh.nv) {                                                      \
        case 1: return CALL(1, 256);                                      \
        case 2: return CALL(2, 256);                                      \
        default: break;                                                   \
    }                                                                     \
    if constexpr (VEC == 4) return CALL(4, 256);                          \
    if constexpr (VEC == 1) {                                             \
        switch (sh.nv) {                                                  \
            case 3: return CALL(3, 256);                                  \
            case 4: return CALL(4, 256);                                  \
            case 5: return CALL(5, 256);                                  \
            case 6: return CALL(6, 256);                                  \
            case 7: return CALL(7, 256);                                  \
            case 8: return CALL(8, 256);                                  \
            default: break;                                               \
        }                                                                 \
    }                                                                     \
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

// vec: elements a vector: 8 (bf16), 4 or 1
cudaError_t launch_ln_fwd(int dtype, int vec, const void* x, const void* res, const float* w,
                          const float* b, void* y, void* sum, float* mean, float* rstd, int64_t N,
                          int64_t D, float eps, cudaStream_t s) {
    if (dtype == 0)
        return vec == 4 ? ln_fwd_t<float, 4>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s)
                        : ln_fwd_t<float, 1>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s);
    return vec == 8   ? ln_fwd_t<__nv_bfloat16, 8>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s)
           : vec == 4 ? ln_fwd_t<__nv_bfloat16, 4>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s)
                      : ln_fwd_t<__nv_bfloat16, 1>(x, res, w, b, y, sum, mean, rstd, N, D, eps, s);
}

cudaError_t launch_ln_bwd(int dtype, int vec, const void* x, const float* w, const float* mean,
                          const float* rstd, const void* dy, const void* dres, void* dx, float* dw,
                          float* db, float* partials, int64_t N, int64_t D, cudaStream_t s) {
    if (dtype == 0)
        return vec == 4 ? ln_bwd_t<float, 4>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s)
                        : ln_bwd_t<float, 1>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s);
    return vec == 8   ? ln_bwd_t<__nv_bfloat16, 8>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s)
           : vec == 4 ? ln_bwd_t<__nv_bfloat16, 4>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s)
                      : ln_bwd_t<__nv_bfloat16, 1>(x, w, mean, rstd, dy, dres, dx, dw, db, partials, N, D, s);
}

}  // namespace lrs
