// lce_kernels.cu -- softmax cross entropy of the logits x W^T over a large
// vocabulary, in pieces of the vocabulary, without keeping the logits.
//
//   l[n][v] = sum_d x[n][d] W[v][d],   lse[n] = log sum_v exp l[n][v],
//   loss[n] = lse[n] - l[n][target[n]]   (0 on ignored rows),
//   g[n][v] = (exp(l[n][v] - lse[n]) - [v = target[n]]) dloss[n],
//   dx = g W,   dW = g^T x.
//
// Forward: a tile of logits lives in registers; each leaves, per row, its
// maximum and its sum of exponentials relative to that maximum, and a second
// kernel joins the tiles' pairs.  Backward: for a piece of the vocabulary the
// logits are computed again and g is written, then the piece's dW and its share
// of dx (summed over the pieces in fp32).
#include "lr_launch.h"

namespace lrs {

namespace {

constexpr int kT = 64, kK = 16;  // tile edge, depth of a step

__device__ __forceinline__ float ldf(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// C[m][n] = sum_k A[m*am + k*ak] B[n*bn + k*bk] over one 64 x 64 tile, 4 x 4 a
// thread (rows ty + 16 i, columns tx + 16 j), handed to the epilogue.
template <typename TA, typename TB, class Epi>
__device__ __forceinline__ void tile_mm(const TA* A, int64_t am, int64_t ak, const TB* B, int64_t bn, int64_t bk,
                                        int64_t M, int64_t N, int64_t K, int64_t m0, int64_t n0, Epi epi) {
    __shared__ float sa[kK][kT + 1], sb[kK][kT + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kK) {
        for (int i = threadIdx.x; i < kT * kK; i += 256) {
            // neighbouring threads along the contiguous axis
            const int ma = ak == 1 ? i / kK : i % kT, ka = ak == 1 ? i % kK : i / kT;
            const int nb = bk == 1 ? i / kK : i % kT, kb = bk == 1 ? i % kK : i / kT;
            sa[ka][ma] = m0 + ma < M && k0 + ka < K ? ldf(A + (m0 + ma) * am + (k0 + ka) * ak) : 0.f;
            sb[kb][nb] = n0 + nb < N && k0 + kb < K ? ldf(B + (n0 + nb) * bn + (k0 + kb) * bk) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { a[i] = sa[k][ty + 16 * i]; b[i] = sb[k][tx + 16 * i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
    epi(acc, m0 + ty, n0 + tx);
}

template <typename S>
__global__ void __launch_bounds__(256)
    k_lce_stats(const S* x, const S* w, const int64_t* target, float2* part, float* tl, int64_t N, int64_t V, int64_t D) {
    const int64_t m0 = (int64_t)blockIdx.y * kT, n0 = (int64_t)blockIdx.x * kT;
    tile_mm(x, D, 1, w, D, 1, N, V, D, m0, n0, [&](float (&acc)[4][4], int64_t m, int64_t n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = m + 16 * i;
            const int64_t t = row < N ? target[row] : -1;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + 16 * j < V) {
                    top = fmaxf(top, acc[i][j]);
                    if (n + 16 * j == t) tl[row] = acc[i][j];
                }
            for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + 16 * j < V) sum += expf(acc[i][j] - top);
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (row < N && (threadIdx.x & 15) == 0) part[(int64_t)blockIdx.x * N + row] = make_float2(top, sum);
        }
    });
}

__global__ void __launch_bounds__(256)
    k_lce_join(const float2* part, int64_t tiles, const float* tl, const int64_t* target, int64_t ignore, float* loss,
               float* lse, int64_t N, int64_t V, uint32_t* err) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float top = -INFINITY, sum = 0.f;
    for (int64_t k = 0; k < tiles; ++k) top = fmaxf(top, part[k * N + n].x);
    for (int64_t k = 0; k < tiles; ++k) sum += part[k * N + n].y * expf(part[k * N + n].x - top);
    const float z = top + logf(sum);
    lse[n] = z;
    const int64_t t = target[n];
    const bool in = t >= 0 && t < V;
    if (!in && t != ignore) atomicOr(err, ERRBIT_INDEX);
    loss[n] = t == ignore || !in ? 0.f : z - tl[n];
}

template <typename S>
__global__ void __launch_bounds__(256)
    k_lce_grad(const S* x, const S* w, const int64_t* target, int64_t ignore, const float* lse, const float* dloss,
               float* g, int64_t N, int64_t v0, int64_t vc, int64_t V, int64_t D) {
    const int64_t m0 = (int64_t)blockIdx.y * kT, n0 = (int64_t)blockIdx.x * kT;
    tile_mm(x, D, 1, w + v0 * D, D, 1, N, vc, D, m0, n0, [&](float (&acc)[4][4], int64_t m, int64_t n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = m + 16 * i;
            if (row >= N) continue;
            const int64_t t = target[row];
            const float s = t == ignore || t < 0 || t >= V ? 0.f : dloss[row];
            const float z = lse[row];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + 16 * j < vc)
                    // the target's p - 1 without cancellation where p is near 1
                    g[row * vc + n + 16 * j] =
                        s == 0.f ? 0.f : (v0 + n + 16 * j == t ? expm1f(acc[i][j] - z) : expf(acc[i][j] - z)) * s;
        }
    });
}

// dx: out[n][d] (+)= sum over the piece; the last piece rounds to the storage type
template <typename S>
__global__ void __launch_bounds__(256)
    k_lce_dx(const float* g, const S* w, float* acc32, S* dx, int64_t N, int64_t v0, int64_t vc, int64_t D, bool first,
             bool last) {
    tile_mm(g, vc, 1, w + v0 * D, 1, D, N, D, vc, (int64_t)blockIdx.y * kT, (int64_t)blockIdx.x * kT,
            [&](float (&acc)[4][4], int64_t m, int64_t n) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t row = m + 16 * i, col = n + 16 * j;
                        if (row >= N || col >= D) continue;
                        const float s = acc[i][j] + (first ? 0.f : acc32[row * D + col]);
                        if (last) {
                            const float o[1] = {s};
                            store_vec<S, 1>(dx + row * D + col, o);
                        } else {
                            acc32[row * D + col] = s;
                        }
                    }
            });
}

template <typename S>
__global__ void __launch_bounds__(256)
    k_lce_dw(const float* g, const S* x, S* dw, int64_t N, int64_t v0, int64_t vc, int64_t D) {
    tile_mm(g, 1, vc, x, 1, D, vc, D, N, (int64_t)blockIdx.y * kT, (int64_t)blockIdx.x * kT,
            [&](float (&acc)[4][4], int64_t m, int64_t n) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t row = m + 16 * i, col = n + 16 * j;
                        const float o[1] = {acc[i][j]};
                        if (row < vc && col < D) store_vec<S, 1>(dw + (v0 + row) * D + col, o);
                    }
            });
}

template <typename S>
cudaError_t lce_fwd_t(const void* x, const void* w, const int64_t* target, int64_t ignore, float* loss, float* lse,
                      int64_t N, int64_t V, int64_t D, const LcePlan& pl, void* scratch, uint32_t* err, cudaStream_t s) {
    float2* part = (float2*)scratch;
    float* tl = (float*)(part + pl.tiles * pl.rows);
    for (int64_t r = 0; r < N; r += pl.rows) {
        const int64_t n = N - r < pl.rows ? N - r : pl.rows;
        k_lce_stats<S><<<dim3((unsigned)pl.tiles, (unsigned)((n + kT - 1) / kT)), 256, 0, s>>>(
            (const S*)x + r * D, (const S*)w, target + r, part, tl, n, V, D);
        k_lce_join<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(part, pl.tiles, tl, target + r, ignore, loss + r, lse + r,
                                                               n, V, err);
    }
    return cudaGetLastError();
}

template <typename S>
cudaError_t lce_bwd_t(const void* x, const void* w, const int64_t* target, int64_t ignore, const float* lse,
                      const float* dloss, void* dx, void* dw, int64_t N, int64_t V, int64_t D, const LcePlan& pl,
                      void* scratch, cudaStream_t s) {
    float* g = (float*)scratch;
    float* acc = g + N * pl.piece;
    for (int64_t v0 = 0; v0 < V; v0 += pl.piece) {
        const int64_t vc = V - v0 < pl.piece ? V - v0 : pl.piece;
        const unsigned tn = (unsigned)((N + kT - 1) / kT), tv = (unsigned)((vc + kT - 1) / kT),
                       td = (unsigned)((D + kT - 1) / kT);
        k_lce_grad<S><<<dim3(tv, tn), 256, 0, s>>>((const S*)x, (const S*)w, target, ignore, lse, dloss, g, N, v0, vc, V, D);
        k_lce_dx<S><<<dim3(td, tn), 256, 0, s>>>(g, (const S*)w, acc, (S*)dx, N, v0, vc, D, v0 == 0, v0 + vc == V);
        k_lce_dw<S><<<dim3(td, tv), 256, 0, s>>>(g, (const S*)x, (S*)dw, N, v0, vc, D);
    }
    return cudaGetLastError();
}

}  // namespace

LcePlan lce_plan(int dtype, int64_t N, int64_t V, int64_t D) {
    (void)dtype;
    LcePlan p;
    p.tiles = (V + kT - 1) / kT;
    p.rows = N < 16384 ? N : 16384;
    p.piece = V < 8192 ? V : 8192;
    p.fwd_bytes = (size_t)(p.tiles * p.rows) * 8 + (size_t)p.rows * 4;
    p.bwd_bytes = (size_t)(N * p.piece) * 4 + (size_t)(N * D) * 4;
    return p;
}

cudaError_t launch_lce_fwd(int dtype, const void* x, const void* w, const int64_t* target, int64_t ignore, float* loss,
                           float* lse, int64_t N, int64_t V, int64_t D, const LcePlan& pl, void* scratch, uint32_t* err,
                           cudaStream_t s) {
    return dtype == 0 ? lce_fwd_t<float>(x, w, target, ignore, loss, lse, N, V, D, pl, scratch, err, s)
                      : lce_fwd_t<__nv_bfloat16>(x, w, target, ignore, loss, lse, N, V, D, pl, scratch, err, s);
}

cudaError_t launch_lce_bwd(int dtype, const void* x, const void* w, const int64_t* target, int64_t ignore,
                           const float* lse, const float* dloss, void* dx, void* dw, int64_t N, int64_t V, int64_t D,
                           const LcePlan& pl, void* scratch, uint32_t* err, cudaStream_t s) {
    (void)err;
    return dtype == 0 ? lce_bwd_t<float>(x, w, target, ignore, lse, dloss, dx, dw, N, V, D, pl, scratch, s)
                      : lce_bwd_t<__nv_bfloat16>(x, w, target, ignore, lse, dloss, dx, dw, N, V, D, pl, scratch, s);
}

}  // namespace lrs
