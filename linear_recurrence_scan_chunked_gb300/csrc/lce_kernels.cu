// lce_kernels.cu -- softmax cross entropy of the logits x W^T over a large
// vocabulary, in pieces of the vocabulary, without keeping the logits.
//
//   l[n][v] = sum_d x[n][d] W[v][d],   lse[n] = log sum_v exp l[n][v],
//   loss[n] = lse[n] - l[n][target[n]]   (0 on ignored rows),
//   g[n][v] = (exp(l[n][v] - lse[n]) - [v = target[n]]) dloss[n],
//   dx = g W,   dW = g^T x.
//
// Forward: the epilogue of the product x W^T reduces each 128 columns of
// logits to a pair per row, their largest M and the sum of exp(l - M), and a second
// kernel joins the tiles' pairs.  Backward:
// for a piece of the vocabulary the product runs again, its epilogue writes g
// (scratch, bounded by kPieceBytes), and two more products give the piece's dW and
// its share of dx, which is added onto one fp32 sum where there are several pieces.
// That is 8 N V D operations where a form that kept the logits needs 6, but no N x V
// array past the budget.
//
// Types.  g is held in bf16 for bf16 data: relative error 2^-9 an element,
// independent from element to element, as much as the rounding of the results.
// It is scaled by 1 / max|dloss| (put back in fp32 at the end), so that with a
// uniform dloss the -1 of the targets is exact and no common rounding error adds
// up in dW.  fp32 data runs as three bf16 planes (lce_mma.cuh), g included.  All
// sums and statistics are fp32.
//
// No floating-point atomics: sums over parts of the k loop are stored as parts and
// added in order.
//
// Measured (cuBLAS bf16 1.92 PFLOP/s in a burst, 1.71 sustained).  bf16 8192 x 1024,
// V 65536, loss and gradients: 2.93 to 3.02 ms over boxes (power capped), 1.50 to
// 1.46 PFLOP/s over the 8 N V D; each product from cold: logits 696 us, their gradient
// 716, dx 665, dW 703, the rest 42.  Loss alone, 4096 x 4096, V 131072: 2.76 to 2.80 ms,
// 1.59 to 1.57 PFLOP/s.  fp32 509 x 250, V 10007: 113 us in eight launches, the
// largest 33, none of which fills the GPU for long.
#include <algorithm>
#include <utility>

#include "lce_mma.cuh"
#include "lr_act.cuh"
#include "lr_launch.h"

namespace lrs {

namespace {

using mm::kTile;
using mm::Shape;
using mm::Tile;

constexpr int64_t kPieceBytes = (int64_t)2 << 30;  // g of one piece, all planes
// k-blocks of a chunk of dx and dW, bf16 data.  8192 x 1024, V 65536, and the mean error
// of dx over 131072 words whose terms have one sign: 16 2963 us, 32 2928 us and 8e-6,
// 64 2916 us and 1.5e-5, one accumulator 2892 us and 7e-4 (the results' rounding: 1e-3
// of each, but with either sign).
constexpr uint32_t kSumChunk = 32;

// 32 bytes of a row (sm_100+: one sector in one store).
__device__ __forceinline__ void st_32b(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// 32 consecutive elements of a row, the first n of them inside it; wide: p is
// 32-byte aligned.
__device__ __forceinline__ void st_row32(__nv_bfloat16* p, const float (&v)[32], int64_t n, bool wide) {
    if (wide && n >= 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = bf_pack(v[16 * h + 2 * i], v[16 * h + 2 * i + 1]);
            st_32b(p + 16 * h, w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
}
__device__ __forceinline__ void st_row32(float* p, const float (&v)[32], int64_t n, bool wide) {
    if (wide && n >= 32) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
            st_32b(p + 8 * h, w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) p[i] = v[i];
    }
}

// v[j] of a runtime j, by selection (the array stays in registers).
__device__ __forceinline__ float pick32(const float (&v)[32], int j) {
    float r = v[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) r = i == j ? v[i] : r;
    return r;
}

// 2^(x log2 e), and what a sum of exponentials relative to `from` is worth relative to
// `to` (infinite ones included: a tile that holds nothing has from = -inf).
__device__ __forceinline__ float exp_fast(float x) { return ex2_ftz(x * kLog2e); }
__device__ __forceinline__ float rescale(float from, float to) { return from == to ? 1.f : exp_fast(from - to); }

// Forward: the pair of a tile and a row, M = max l and the sum of e^(l - M).  The
// difference is taken before it is scaled, so that logits of any finite size keep
// their places, words masked by the type's lowest value count as 0 and only a NaN or
// +inf logit makes the sum NaN or infinite.
template <bool CHUNKED, int P>
struct StatsEpi {
    static constexpr bool kChunked = CHUNKED, kStaged = false;
    static constexpr int kPlanes = P;
    static constexpr uint32_t kChunk = mm::chunk_of(P);
    float2* part;           // [half tiles][rows]
    float* tl;              // the targets' logits
    const int64_t* target;
    int64_t rows, V;
    int tn;                 // columns of a tile
    struct Row {
        int64_t n, slot;
        int width, at;
        float M, s;
    };
    __device__ int width(const Tile& t, int half) const {
        const int64_t w = V - ((int64_t)t.n * 2 + half) * (tn / 2);
        return (int)(w < tn / 2 ? w : tn / 2);
    }
    __device__ Row begin(const Tile& t, int row, int half) const {
        Row r;
        r.n = (int64_t)t.m * kTile + row;
        r.slot = (int64_t)t.n * 2 + half;
        r.width = width(t, half);
        const int64_t tg = r.n < rows ? __ldg(target + r.n) - r.slot * (tn / 2) : -1;
        r.at = tg >= 0 && tg < r.width ? (int)tg : -1;
        r.M = -INFINITY;
        r.s = 0.f;
        return r;
    }
    __device__ void cols(Row& r, int c, float (&v)[32], float*) const {
        if (r.width < c * 32 + 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = c * 32 + i < r.width ? v[i] : -INFINITY;
        }
        if (__any_sync(0xffffffffu, r.at >> 5 == c)) {
            const float x = pick32(v, r.at & 31);
            if (r.at >> 5 == c) tl[r.n] = x;
        }
        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int i = 4; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], v[i]);
        const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (m > r.M) {
            r.s *= exp_fast(r.M - m);  // the first time e^-inf = 0
            r.M = m;
        }
        // nothing but -inf so far, or a +inf: their own exponentials
        const float base = fabsf(r.M) < INFINITY ? r.M : 0.f;
        float e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) e[i & 3] += exp_fast(v[i] - base);
        r.s += (e[0] + e[1]) + (e[2] + e[3]);
    }
    __device__ void end(Row& r) const {
        if (r.n < rows && r.width > 0) part[r.slot * rows + r.n] = make_float2(r.M, r.s);
    }
};

// Joins the tiles' pairs of 32 rows (x): lane y folds tiles y, y + 32, ..., then
// the lanes' pairs fold in order.
__global__ void __launch_bounds__(1024)
    k_lce_join(const float2* __restrict__ part, int64_t tiles, const float* __restrict__ tl,
               const int64_t* __restrict__ target, int64_t ignore, float* __restrict__ loss, float* __restrict__ lse,
               int64_t rows, int64_t V, uint32_t* err) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float2 sm[32][33];
    const int64_t n = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float M = -INFINITY, s = 0.f;
    auto fold = [&](const float2 p) {
        const float m = fmaxf(M, p.x);
        s = s * rescale(M, m) + p.y * rescale(p.x, m);
        M = m;
    };
    if (n < rows) {
        int64_t k = threadIdx.y;
        for (; k + 224 < tiles; k += 256) {  // eight loads in flight
            float2 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = __ldg(part + (k + 32 * u) * rows + n);
#pragma unroll
            for (int u = 0; u < 8; ++u) fold(v[u]);
        }
#pragma unroll 4
        for (; k < tiles; k += 32) fold(__ldg(part + k * rows + n));
    }
    sm[threadIdx.y][threadIdx.x] = make_float2(M, s);
    __syncthreads();
    if (threadIdx.y != 0 || n >= rows) return;
    M = -INFINITY;
    s = 0.f;
    for (int k = 0; k < 32 && k < tiles; ++k) fold(sm[k][threadIdx.x]);
    const float z = M + logf(s);
    lse[n] = z;
    const int64_t t = target[n];
    const bool in = t >= 0 && t < V;
    if (!in && t != ignore) atomicOr(err, ERRBIT_INDEX);
    loss[n] = t == ignore || !in ? 0.f : z - tl[n];
}

__device__ __forceinline__ float scale_of(const uint32_t* top) {
    const float s = __uint_as_float(__ldg(top));
    return s > 0.f ? s : 1.f;
}

// Backward: g / max|dloss| of a tile, in P bf16 planes.  Its logits are the forward
// pass's to the last bit (the k loop in the same chunks): p - 1 of a confident row is
// the difference of a logit and lse, which then are off by the same.  (One accumulator
// over k = 4096 here, chunks there: a gradient at p = 0.999 came out 19% off.)
template <bool CHUNKED, int P>
struct GradEpi {
    static constexpr bool kChunked = CHUNKED, kStaged = false;
    static constexpr int kPlanes = P;
    static constexpr uint32_t kChunk = mm::chunk_of(P);
    __nv_bfloat16* g;  // [P][rows][pitch]
    int64_t pitch;     // a multiple of 16
    int64_t plane;     // elements of a plane
    const float* lse;
    const float* dloss;
    const int64_t* target;
    const uint32_t* top;
    int64_t ignore, rows, v0, vc, V;
    int tn;
    struct Row {
        int64_t n;
        __nv_bfloat16* out;
        int width, at;
        bool live;      // the row counts
        float ds, z;
    };
    __device__ int width(const Tile& t, int half) const {
        const int64_t w = vc - ((int64_t)t.n * 2 + half) * (tn / 2);
        return (int)(w < tn / 2 ? w : tn / 2);
    }
    __device__ Row begin(const Tile& t, int row, int half) const {
        Row r;
        r.n = (int64_t)t.m * kTile + row;
        const int64_t c0 = ((int64_t)t.n * 2 + half) * (tn / 2);
        r.width = width(t, half);
        r.out = g + r.n * pitch + c0;
        r.ds = r.z = 0.f;
        r.live = false;
        r.at = -1;
        if (r.n < rows) {
            const int64_t tg = __ldg(target + r.n);
            if (tg != ignore && tg >= 0 && tg < V) {
                r.ds = __fdiv_rn(__ldg(dloss + r.n), scale_of(top));
                r.z = __ldg(lse + r.n);
                r.live = true;
                const int64_t q = tg - v0 - c0;
                if (q >= 0 && q < r.width) r.at = (int)q;
            }
        }
        return r;
    }
    __device__ void cols(Row& r, int c, float (&v)[32], float*) const {
        const bool mine = r.at >> 5 == c, any = __any_sync(0xffffffffu, mine);
        float gt = 0.f;
        // the target's p - 1 without cancellation where p is near 1
        if (any) gt = expm1f(pick32(v, r.at & 31) - r.z) * r.ds;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = exp_fast(v[i] - r.z) * r.ds;
        if (!r.live) {  // whatever its logits are, infinite or NaN
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        if (any) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = mine && i == (r.at & 31) ? gt : v[i];
        }
        if (r.n >= rows) return;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            st_row32(r.out + p * plane + c * 32, v, r.width - c * 32, true);
            if (p + 1 < P) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] -= bf_lo(bf_bits(v[i]));
            }
        }
    }
    __device__ void end(Row&) const {}
};

// A product's tile: rounded to the result (scaled by max|dloss|), or one part of
// the k loop, fp32.
template <bool CHUNKED, typename S>
struct OutEpi {
    static constexpr bool kChunked = CHUNKED, kStaged = true;
    static constexpr int kPlanes = sizeof(S) == 4 ? 3 : 1;
    static constexpr uint32_t kChunk = kPlanes == 1 ? kSumChunk : mm::chunk_of(kPlanes);
    S* out;         // nullptr: parts
    float* part;    // [splits][rows x cols]
    int64_t pitch;  // elements of a part
    const uint32_t* top;
    int64_t rows, cols_n;
    int tn;
    bool wide;      // rows of the destination are 32-byte aligned
    struct Row {
        int64_t m, at;
        int width;
        float a;
    };
    __device__ int width(const Tile& t, int half) const {
        const int64_t w = cols_n - ((int64_t)t.n * 2 + half) * (tn / 2);
        return (int)(w < tn / 2 ? w : tn / 2);
    }
    __device__ Row begin(const Tile& t, int row, int half) const {
        Row r;
        r.m = (int64_t)t.m * kTile + row;
        r.width = width(t, half);
        r.at = (out ? 0 : t.split * pitch) + r.m * cols_n + ((int64_t)t.n * 2 + half) * (tn / 2);
        r.a = out ? scale_of(top) : 1.f;
        return r;
    }
    __device__ void cols(Row& r, int c, float (&v)[32], float* scratch) const {
        if (out) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= r.a;
        }
        if (wide && r.width - c * 32 >= 32) {  // 32 bytes a lane, whole sectors
            if (r.m >= rows) return;
            if (out) st_row32(out + r.at + c * 32, v, 32, true);
            else st_row32(part + r.at + c * 32, v, 32, true);
            return;
        }
        // unaligned rows: through shared memory, so that a store writes 32
        // neighbouring elements of one row
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 32; ++i) scratch[lane * 33 + i] = v[i];
        __syncwarp();
        const int64_t m0 = r.m - lane, at0 = r.at - lane * cols_n + c * 32 + lane;
        const int n = (int)(rows - m0 < 32 ? rows - m0 : 32);
        if (lane < r.width - c * 32) {
            for (int i = 0; i < n; ++i) {
                const float o[1] = {scratch[i * 33 + lane]};
                if (out) store_vec<S, 1>(out + at0 + i * cols_n, o);
                else store_vec<float, 1>(part + at0 + i * cols_n, o);
            }
        }
        __syncwarp();
    }
    __device__ void end(Row&) const {}
};

// out = scale * (add + the sum of the parts), scale = max|dloss| or, without `top`, 1;
// add (nullptr: none): fp32, may be `out` itself.  GROUPS warps share 128 (vec) or 32
// outputs: each adds a run of neighbouring parts in order, and the runs' sums are
// added in order.
template <typename S, int GROUPS>
__global__ void __launch_bounds__(256)
    k_lce_sum(const float* __restrict__ part, int64_t parts, int64_t pitch, int64_t n, const float* add,
              const uint32_t* __restrict__ top, S* out, bool vec) {
    griddep_launch_dependents();
    griddep_wait();
    const float a = top != nullptr ? scale_of(top) : 1.f;
    constexpr int kLanes = 256 / GROUPS;  // threads of a run
    const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    const int64_t step = (int64_t)gridDim.x * kLanes, run = (parts + GROUPS - 1) / GROUPS;
    const int64_t k0 = grp * run, k1 = parts < k0 + run ? parts : k0 + run;
    __shared__ float4 sm[GROUPS > 1 ? 256 : 1];
    auto sum = [&](auto width, int64_t base, int64_t count) {
        constexpr int W = decltype(width)::value;
        for (int64_t i0 = (int64_t)blockIdx.x * kLanes; i0 < count; i0 += step) {
            const int64_t i = i0 + lane;
            float s[W];
#pragma unroll
            for (int j = 0; j < W; ++j) s[j] = 0.f;
            if (i < count) {
                if (add != nullptr && grp == 0) {
#pragma unroll
                    for (int j = 0; j < W; ++j) s[j] = add[base + W * i + j];
                }
                int64_t k = k0;
                for (; k + 8 <= k1; k += 8) {  // eight loads in flight, added in order
                    Pack<float, W> p[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) p[u].load(part + (k + u) * pitch + base + W * i);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
#pragma unroll
                        for (int j = 0; j < W; ++j) s[j] += p[u].get(j);
                }
#pragma unroll 4
                for (; k < k1; ++k) {
                    Pack<float, W> p;
                    p.load(part + k * pitch + base + W * i);
#pragma unroll
                    for (int j = 0; j < W; ++j) s[j] += p.get(j);
                }
            }
            if constexpr (GROUPS > 1) {
                float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
                q.x = s[0];
                if constexpr (W == 4) { q.y = s[1]; q.z = s[2]; q.w = s[3]; }
                __syncthreads();
                sm[threadIdx.x] = q;
                __syncthreads();
                if (grp > 0) continue;
#pragma unroll
                for (int r = 1; r < GROUPS; ++r) {
                    const float4 o = sm[r * kLanes + lane];
                    s[0] += o.x;
                    if constexpr (W == 4) { s[1] += o.y; s[2] += o.z; s[3] += o.w; }
                }
            }
            if (i < count) {
#pragma unroll
                for (int j = 0; j < W; ++j) s[j] *= a;
                store_vec<S, W>(out + base + W * i, s);
            }
        }
    };
    if (vec) sum(std::integral_constant<int, 4>{}, 0, n / 4);
    const int64_t done = vec ? n / 4 * 4 : 0;
    sum(std::integral_constant<int, 1>{}, done, n - done);
}

// bf16's largest number in place of finite ones beyond it.
constexpr float kBfMax = 0x1.fep127f;
__device__ __forceinline__ float bf_bound(float x) {
    return fabsf(x) > kBfMax && fabsf(x) < INFINITY ? copysignf(kBfMax, x) : x;
}

// A matrix on its way into planes: [rows][D] into P bf16 planes of pitch ld (a
// multiple of 8; the columns past D are never read).
struct PackJob {
    const void* src;
    __nv_bfloat16* dst;
    int64_t rows, D, ld;
    int vec;  // elements that can be read at once: 4, 2 or 1
};

// Before the products, one launch: block 0 takes max |dloss| over the rows that
// count (finite ones) into `top`, as float bits; the other blocks pack x and W --
// fp32 data split into three planes, bf16 data whose rows TMA cannot read (odd
// widths, unaligned views) copied.  A warp takes a row, four elements a lane; LONG
// rows (from 512 elements) four times four, whose loads are in flight together
// (bf16 9928 x 2074: 25 -> 16 us; shorter rows pay for the registers: fp32
// 62522 x 261 28 -> 33 us).
template <typename S, int P, bool LONG>
__global__ void __launch_bounds__(256)
    k_lce_prep(const PackJob jx, const PackJob jw, const float* __restrict__ dloss, const int64_t* __restrict__ target,
               int64_t ignore, int64_t N, int64_t V, uint32_t* __restrict__ top) {
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0) {
        __shared__ uint32_t sm[8];
        if (top == nullptr) return;
        uint32_t m = 0;
        for (int64_t n0 = threadIdx.x; n0 < N; n0 += 1024) {
            float a[4];
            int64_t t[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t n = n0 + 256 * u;
                a[u] = n < N ? fabsf(__ldg(dloss + n)) : 0.f;
                t[u] = n < N ? __ldg(target + n) : ignore;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (t[u] != ignore && t[u] >= 0 && t[u] < V && a[u] < INFINITY) m = max(m, __float_as_uint(a[u]));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) sm[warp] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 8; ++w) m = max(m, sm[w]);
            *top = m;
        }
        return;
    }
    const int64_t warps = (int64_t)(gridDim.x - 1) * 8;
    for (int64_t row = (int64_t)(blockIdx.x - 1) * 8 + warp; row < jx.rows + jw.rows; row += warps) {
        const bool first = row < jx.rows;
        const PackJob& j = first ? jx : jw;
        const int64_t r = first ? row : row - jx.rows;
        const S* src = (const S*)j.src + r * j.D;
        __nv_bfloat16* dst = j.dst + r * j.ld;
        const int64_t plane = j.rows * j.ld;
        // rows are padded to 8: 8-byte stores stay inside
        auto put = [&](int64_t d, float (&v)[4]) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                uint32_t a = bf_pack(v[0], v[1]), b = bf_pack(v[2], v[3]);
                if constexpr (P > 1) {
                    // past bf16's largest number the first plane is that number, not infinite
                    const float t = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
                    if (k == 0 && t > kBfMax) {
                        a = bf_pack(bf_bound(v[0]), bf_bound(v[1]));
                        b = bf_pack(bf_bound(v[2]), bf_bound(v[3]));
                    }
                }
                *reinterpret_cast<uint2*>(dst + k * plane + d) = make_uint2(a, b);
                v[0] -= bf_lo(a); v[1] -= bf_hi(a); v[2] -= bf_lo(b); v[3] -= bf_hi(b);
            }
        };
        auto get = [&](auto width, int64_t d, float (&v)[4]) {
            constexpr int W = decltype(width)::value;
#pragma unroll
            for (int i = 0; i < 4; i += W) {
                Pack<S, W> p;
                p.load(src + d + i);
#pragma unroll
                for (int k = 0; k < W; ++k) v[i + k] = p.get(k);
            }
        };
        int64_t d = lane * 4;
        if constexpr (LONG) {
            auto bulk = [&](auto width) {  // four quads in flight
                for (; d + 384 + 4 <= j.D; d += 512) {
                    float v[4][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) get(width, d + 128 * q, v[q]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) put(d + 128 * q, v[q]);
                }
            };
            if (j.vec == 4) bulk(std::integral_constant<int, 4>{});
            else if (j.vec == 2) bulk(std::integral_constant<int, 2>{});
            else bulk(std::integral_constant<int, 1>{});
        }
        for (; d < j.D; d += 128) {
            float v[4];
            if (j.vec == 4) {
                get(std::integral_constant<int, 4>{}, d, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Pack<S, 1> p;
                    p.ident(0.f);
                    if (d + i < j.D) p.load(src + d + i);
                    v[i] = p.get(0);
                }
            }
            put(d, v);
        }
    }
}

// ------------------------------------------------------------------- host
//
// Every kernel of a call is launched by launch_dep and waits for the one before it
// (griddep_wait) before it touches memory.

// An operand as the products take it: bf16 planes [planes][rows][ld].
struct Operand {
    const __nv_bfloat16* p;
    int64_t rows, cols, ld, plane;
    int planes;
};

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// mn: the product takes it MN-major (boxes of 64 x 64), else K-major (64 x box_rows).
bool operand_map(CUtensorMap* m, const Operand& o, bool mn, int box_rows) {
    return tma_encode_planes(m, o.p, o.cols, o.rows, o.planes, o.ld, o.plane, mm::kBlockK, mn ? mm::kBlockK : box_rows);
}

// Pairs of CTAs resident at once.
template <class Epi, int TN>
cudaError_t mm_pairs(int* pairs) {
    static int known[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    int& n = known[dev & 63];
    constexpr int smem = mm::Cfg<TN>::smem(Epi::kStaged);
    if (n <= 0) {
        cudaError_t e = cudaFuncSetAttribute(mm::k_mm<Epi, TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t lc{};
        lc.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
        lc.blockDim = dim3(mm::kThreads);
        lc.dynamicSmemBytes = smem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        lc.attrs = at;
        lc.numAttrs = 1;
        int c = 0;
        if (cudaOccupancyMaxActiveClusters(&c, mm::k_mm<Epi, TN>, &lc) != cudaSuccess || c < 1) c = 1;
        n = c < sm_count() / 2 ? c : sm_count() / 2;
    }
    *pairs = n;
    return cudaSuccess;
}

template <class Epi, int TN>
cudaError_t mm_launch(const Operand& a, const Operand& b, const Shape& sh, const Epi& epi, uint32_t* err, cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!operand_map(&ma, a, sh.a_mn, mm::kHalf) || !operand_map(&mb, b, sh.b_mn, TN / 2)) return cudaErrorInvalidValue;
    int pairs = 1;
    const cudaError_t e = mm_pairs<Epi, TN>(&pairs);
    if (e != cudaSuccess) return e;
    const uint64_t tiles = (uint64_t)sh.tm * sh.tn * sh.splits;
    if (tiles > 0x7fffffffull) return cudaErrorInvalidValue;
    const unsigned grid = 2 * (unsigned)std::min<uint64_t>(tiles, (uint64_t)pairs);
    return launch_dep(mm::k_mm<Epi, TN>, dim3(grid), dim3(mm::kThreads), mm::Cfg<TN>::smem(Epi::kStaged), s, ma, mb, sh, epi,
                      err);
}

// How a product M x N x K is cut: tiles of 256 x tn, the k loop in `splits` parts.
struct MmPlan {
    int tn;
    int64_t splits;
};

Shape mm_shape(int64_t M, int64_t N, int64_t K, bool a_mn, bool b_mn, bool n_fast, const MmPlan& pl, uint64_t stall_ns) {
    Shape s{};
    s.tm = (uint32_t)((M + kTile - 1) / kTile);
    s.tn = (uint32_t)((N + pl.tn - 1) / pl.tn);
    s.kb = (uint32_t)((K + mm::kBlockK - 1) / mm::kBlockK);
    s.kb_split = (uint32_t)((s.kb + pl.splits - 1) / pl.splits);
    s.splits = (s.kb + s.kb_split - 1) / s.kb_split;
    s.n_fast = n_fast;
    s.a_mn = a_mn;
    s.b_mn = b_mn;
    s.wait_ns = stall_ns ? stall_ns : kMbarLimitNs;
    s.stalled = stall_ns != 0;
    return s;
}

template <class Epi>
cudaError_t mm_run(const Operand& a, const Operand& b, const Shape& sh, Epi epi, int tn, uint32_t* err, cudaStream_t s) {
    epi.tn = tn;
    if constexpr (!Epi::kStaged) {  // the logits: B is K-major
        if (tn == 64) return mm_launch<Epi, 64>(a, b, sh, epi, err, s);
    }
    return tn == 256 ? mm_launch<Epi, 256>(a, b, sh, epi, err, s) : mm_launch<Epi, 128>(a, b, sh, epi, err, s);
}

// The cut of a product that takes the shortest time in a simple model: rounds of
// tiles over the pairs, each at a pair's rate (a k-block of 64 by 256 columns takes
// about 512 cycles, by 128 about 300, by 64 about 190: A comes from L2 more often)
// plus about 1500 cycles of latency, plus, with more than one part, the parts' way
// to memory and back (about 3.5 KB a cycle over the GPU).  With few tiles narrow ones
// and parts fill the GPU; with many, parts even out its last round.  (fp32 509 x 250,
// V 10007, loss and gradients: 195 us with 256-column tiles only, 160 with the
// choice between 256 and 128, before the other steps.)
MmPlan mm_plan(int64_t M, int64_t N, int64_t K, int planes, bool may_split) {
    const int64_t kb = (K + mm::kBlockK - 1) / mm::kBlockK, pairs = kSpanSms / 2;
    MmPlan best{256, 1};
    double best_t = 0;
    for (int tn : {256, 128, 64}) {
        if (tn == 64 && may_split) break;  // MN-major B: blocks of 64 a CTA
        const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + tn - 1) / tn);
        for (int64_t s = 1; s <= (may_split ? 64 : 1) && s <= kb; ++s) {
            const int64_t per = (kb + s - 1) / s, real = (kb + per - 1) / per;
            if (real != s) continue;
            const double rounds = (double)((tiles * s + pairs - 1) / pairs);
            double t = rounds * ((double)per * (planes == 1 ? 1 : 6) * (tn == 256 ? 512 : tn == 128 ? 300 : 190) + 1500);
            if (s > 1) t += (double)(s * M * N) * 8 / 3500 + 4000;
            if (best_t == 0 || t < 0.98 * best_t) {
                best = MmPlan{tn, s};
                best_t = t;
            }
        }
    }
    return best;
}

struct Layout {  // offsets into the scratch
    size_t x, w, top, part, tl, g, px, acc, pw, bytes;
};

bool packed(int dtype, const void* p, int64_t D) { return dtype == 0 || D % 8 != 0 || ((uintptr_t)p & 15) != 0; }

size_t take(size_t& at, size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
}

Layout layout(int dtype, const void* x, const void* w, int64_t N, int64_t V, int64_t D, const LcePlan& p, bool bwd) {
    Layout l{};
    const size_t planes = dtype == 0 ? 3 : 1;
    const int64_t ld = round_up(D, 8);
    size_t at = 0;
    l.top = take(at, 4);
    if (packed(dtype, x, D)) l.x = take(at, planes * N * ld * 2);
    if (packed(dtype, w, D)) l.w = take(at, planes * V * ld * 2);
    if (bwd) {
        l.g = take(at, planes * N * round_up(p.piece, 16) * 2);
        if (p.dx_splits > 1 || p.piece < V) l.px = take(at, (size_t)p.dx_splits * round_up(N * D, 8) * 4);
        if (dtype == 1 && p.piece < V) l.acc = take(at, (size_t)(N * D) * 4);
        if (p.dw_splits > 1) l.pw = take(at, (size_t)p.dw_splits * round_up(p.piece * D, 8) * 4);
    } else {
        l.part = take(at, (size_t)(p.tiles * p.rows) * 8);
        l.tl = take(at, (size_t)p.rows * 4);
    }
    l.bytes = at;
    return l;
}

// The operand of a caller's matrix, and the job that packs it into the scratch
// where it has to be (rows = 0: it need not).
template <typename S>
Operand operand(const void* src, int64_t rows, int64_t D, void* scratch, PackJob* job) {
    constexpr int P = sizeof(S) == 4 ? 3 : 1;
    *job = PackJob{nullptr, nullptr, 0, 0, 0, 1};
    if (!packed(sizeof(S) == 4 ? 0 : 1, src, D)) return Operand{(const __nv_bfloat16*)src, rows, D, D, rows * D, P};
    const int64_t ld = round_up(D, 8);
    int vec = 4;
    while (vec > 1 && (D % vec != 0 || ((uintptr_t)src & (vec * sizeof(S) - 1)) != 0)) vec /= 2;
    *job = PackJob{src, (__nv_bfloat16*)scratch, rows, D, ld, vec};
    return Operand{(const __nv_bfloat16*)scratch, rows, D, ld, rows * ld, P};
}

template <typename S>
cudaError_t prepare(const PackJob& jx, const PackJob& jw, const float* dloss, const int64_t* target, int64_t ignore,
                    int64_t N, int64_t V, uint32_t* top, cudaStream_t s) {
    const int64_t rows = jx.rows + jw.rows;
    if (rows == 0 && top == nullptr) return cudaSuccess;
    const int64_t blocks = 1 + std::min<int64_t>((rows + 7) / 8, (int64_t)sm_count() * 8);
    constexpr int P = sizeof(S) == 4 ? 3 : 1;
    const bool wide = std::max(jx.D, jw.D) >= 512;
    return launch_dep(wide ? k_lce_prep<S, P, true> : k_lce_prep<S, P, false>, dim3((unsigned)blocks), dim3(256), 0, s, jx, jw,
                      dloss, target, ignore, N, V, top);
}

#define LCE_TRY(x)                            \
    do {                                      \
        const cudaError_t e_ = (x);           \
        if (e_ != cudaSuccess) return e_;     \
    } while (0)

template <typename S>
cudaError_t lce_fwd_t(const void* x, const void* w, const int64_t* target, int64_t ignore, float* loss, float* lse,
                      int64_t N, int64_t V, int64_t D, const LcePlan& pl, char* sc, uint32_t* err, cudaStream_t s) {
    const Layout l = layout(sizeof(S) == 4 ? 0 : 1, x, w, N, V, D, pl, false);
    PackJob jx, jw;
    const Operand ox = operand<S>(x, N, D, sc + l.x, &jx), ow = operand<S>(w, V, D, sc + l.w, &jw);
    LCE_TRY(prepare<S>(jx, jw, nullptr, target, ignore, N, V, nullptr, s));
    float2* part = (float2*)(sc + l.part);
    float* tl = (float*)(sc + l.tl);
    for (int64_t r = 0; r < N; r += pl.rows) {
        const int64_t n = std::min(pl.rows, N - r);
        Operand a = ox;
        a.p += r * a.ld;
        a.rows = n;
        const Shape sh = mm_shape(n, V, D, false, false, false, MmPlan{pl.tn_logits, 1}, pl.stall_ns);
        constexpr int P = sizeof(S) == 4 ? 3 : 1;
        if (sh.kb > mm::chunk_of(P))
            LCE_TRY(mm_run(a, ow, sh, StatsEpi<true, P>{part, tl, target + r, n, V, 0}, pl.tn_logits, err, s));
        else
            LCE_TRY(mm_run(a, ow, sh, StatsEpi<false, P>{part, tl, target + r, n, V, 0}, pl.tn_logits, err, s));
        LCE_TRY(launch_dep(k_lce_join, dim3((unsigned)((n + 31) / 32)), dim3(32, 32), 0, s, part, pl.tiles, tl, target + r,
                           ignore, loss + r, lse + r, n, V, err));
    }
    return cudaSuccess;
}

template <typename S>
cudaError_t sum_parts(const float* part, int64_t parts, int64_t pitch, int64_t n, const float* add, const uint32_t* top,
                      S* out, cudaStream_t s) {
    const bool vec = ((uintptr_t)out & (4 * sizeof(S) - 1)) == 0;
    // few outputs: eight warps to a warp's outputs, or the loads of one thread's
    // parts, one round trip for eight, are the time
    const int64_t items = n / (vec ? 4 : 1) + 1, cap = (int64_t)sm_count() * 8;
    const bool few = parts > 8 && items < (int64_t)sm_count() * 512;
    const int64_t lanes = few ? 32 : 256;
    const dim3 grid((unsigned)std::min<int64_t>((items + lanes - 1) / lanes, cap));
    return few ? launch_dep(k_lce_sum<S, 8>, grid, dim3(256), 0, s, part, parts, pitch, n, add, top, out, vec)
               : launch_dep(k_lce_sum<S, 1>, grid, dim3(256), 0, s, part, parts, pitch, n, add, top, out, vec);
}

template <typename S>
cudaError_t lce_bwd_t(const void* x, const void* w, const int64_t* target, int64_t ignore, const float* lse,
                      const float* dloss, void* dx, void* dw, int64_t N, int64_t V, int64_t D, const LcePlan& pl, char* sc,
                      uint32_t* err, cudaStream_t s) {
    constexpr int P = sizeof(S) == 4 ? 3 : 1;
    const Layout l = layout(sizeof(S) == 4 ? 0 : 1, x, w, N, V, D, pl, true);
    uint32_t* top = (uint32_t*)(sc + l.top);
    PackJob jx, jw;
    const Operand ox = operand<S>(x, N, D, sc + l.x, &jx), ow = operand<S>(w, V, D, sc + l.w, &jw);
    LCE_TRY(prepare<S>(jx, jw, dloss, target, ignore, N, V, top, s));
    __nv_bfloat16* g = (__nv_bfloat16*)(sc + l.g);
    float* px = (float*)(sc + l.px);
    float* pw = (float*)(sc + l.pw);
    const int64_t xpitch = round_up(N * D, 8), wpitch = round_up(pl.piece * D, 8);
    const bool wide_s = D * (int64_t)sizeof(S) % 32 == 0, wide_f = D % 8 == 0;
    const uint32_t sum_chunk = OutEpi<true, S>::kChunk;
    // several pieces: dx grows piece by piece, in fp32, in the order of the vocabulary
    const bool pieces = pl.piece < V;
    float* acc = sizeof(S) == 4 ? (float*)dx : (float*)(sc + l.acc);
    for (int64_t v0 = 0; v0 < V; v0 += pl.piece) {
        const int64_t vc = std::min(pl.piece, V - v0), pitch = round_up(vc, 16);
        Operand wp = ow;
        wp.p += v0 * ow.ld;
        wp.rows = vc;
        const Operand og{g, N, vc, pitch, N * pitch, P};
        const Shape sl = mm_shape(N, vc, D, false, false, false, MmPlan{pl.tn_logits, 1}, pl.stall_ns);
        auto logits = [&](auto chunked) {
            return mm_run(ox, wp, sl,
                          GradEpi<decltype(chunked)::value, P>{g, pitch, N * pitch, lse, dloss, target, top, ignore, N, v0, vc, V, 0},
                          pl.tn_logits, err, s);
        };
        LCE_TRY(sl.kb > mm::chunk_of(P) ? logits(std::true_type{}) : logits(std::false_type{}));
        // dx: rows of x by features, over the words of the piece
        const Shape sx = mm_shape(N, D, vc, false, true, true, MmPlan{pl.tn_dx, pl.dx_splits}, pl.stall_ns);
        const bool dx_direct = pl.dx_splits == 1 && !pieces;
        auto dx_of = [&](auto chunked) {
            return mm_run(og, wp, sx,
                          OutEpi<decltype(chunked)::value, S>{dx_direct ? (S*)dx : nullptr, px, xpitch, top, N, D, 0,
                                                              dx_direct ? wide_s && ((uintptr_t)dx & 31) == 0 : wide_f},
                          pl.tn_dx, err, s);
        };
        LCE_TRY(sx.kb_split > sum_chunk ? dx_of(std::true_type{}) : dx_of(std::false_type{}));
        if (!dx_direct) {
            const float* before = v0 > 0 ? acc : nullptr;
            if (v0 + vc < V) LCE_TRY(sum_parts<float>(px, sx.splits, xpitch, N * D, before, nullptr, acc, s));
            else LCE_TRY(sum_parts<S>(px, sx.splits, xpitch, N * D, before, top, (S*)dx, s));
        }
        // dw: words of the piece by features, over the rows of x
        const Shape sw = mm_shape(vc, D, N, true, true, true, MmPlan{pl.tn_dw, pl.dw_splits}, pl.stall_ns);
        const bool dw_direct = pl.dw_splits == 1;
        S* dwp = (S*)dw + v0 * D;
        auto dw_of = [&](auto chunked) {
            return mm_run(og, ox, sw,
                          OutEpi<decltype(chunked)::value, S>{dw_direct ? dwp : nullptr, pw, wpitch, top, vc, D, 0,
                                                              dw_direct ? wide_s && ((uintptr_t)dwp & 31) == 0 : wide_f},
                          pl.tn_dw, err, s);
        };
        LCE_TRY(sw.kb_split > sum_chunk ? dw_of(std::true_type{}) : dw_of(std::false_type{}));
        if (!dw_direct) LCE_TRY(sum_parts<S>(pw, sw.splits, wpitch, vc * D, nullptr, top, dwp, s));
    }
    return cudaSuccess;
}

}  // namespace

LcePlan lce_plan(int dtype, const void* x, const void* w, int64_t N, int64_t V, int64_t D, bool bwd, int64_t budget) {
    LcePlan p{};
    const int planes = dtype == 0 ? 3 : 1;
    if (budget <= 0) budget = kPieceBytes;
    if (!bwd) {
        // rounds of rows whose pairs (of 128 words at least, but for small problems) fit
        p.rows = std::min<int64_t>(std::min<int64_t>(N, 16384), std::max<int64_t>(budget / (V / 128 * 8 + 8) / kTile, 1) * kTile);
        p.tn_logits = mm_plan(p.rows, V, D, planes, false).tn;
        p.tiles = (V + p.tn_logits / 2 - 1) / (p.tn_logits / 2);
    } else {
        p.piece = std::max<int64_t>(budget / (N * 2 * planes) / kTile, 1) * kTile;
        if (p.piece >= V) p.piece = V;
        p.tn_logits = mm_plan(N, p.piece, D, planes, false).tn;
        const MmPlan dx = mm_plan(N, D, p.piece, planes, true), dw = mm_plan(p.piece, D, N, planes, true);
        p.tn_dx = dx.tn;
        p.dx_splits = dx.splits;
        p.tn_dw = dw.tn;
        p.dw_splits = dw.splits;
    }
    p.bytes = layout(dtype, x, w, N, V, D, p, bwd).bytes;
    return p;
}

cudaError_t launch_lce_fwd(int dtype, const void* x, const void* w, const int64_t* target, int64_t ignore, float* loss,
                           float* lse, int64_t N, int64_t V, int64_t D, const LcePlan& pl, void* scratch, uint32_t* err,
                           cudaStream_t s) {
    return dtype == 0 ? lce_fwd_t<float>(x, w, target, ignore, loss, lse, N, V, D, pl, (char*)scratch, err, s)
                      : lce_fwd_t<__nv_bfloat16>(x, w, target, ignore, loss, lse, N, V, D, pl, (char*)scratch, err, s);
}

cudaError_t launch_lce_bwd(int dtype, const void* x, const void* w, const int64_t* target, int64_t ignore,
                           const float* lse, const float* dloss, void* dx, void* dw, int64_t N, int64_t V, int64_t D,
                           const LcePlan& pl, void* scratch, uint32_t* err, cudaStream_t s) {
    return dtype == 0
               ? lce_bwd_t<float>(x, w, target, ignore, lse, dloss, dx, dw, N, V, D, pl, (char*)scratch, err, s)
               : lce_bwd_t<__nv_bfloat16>(x, w, target, ignore, lse, dloss, dx, dw, N, V, D, pl, (char*)scratch, err, s);
}

}  // namespace lrs
