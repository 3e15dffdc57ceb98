// glr_kernels.cu -- gated linear recurrence: the scan h_t = a_t h_{t-1} + b_t
// (page [P1] "CUDA并行化RNN训练：从O(T)到O(log T)的工程实践与参数调优", parallel-scan
// paragraph) with a decay that the input sets and an input scaled so that the
// state keeps its size:
//   r = sigmoid(zr + br),  i = sigmoid(zi + bi),  a = exp(-lam r),  f = sqrt(1 - a^2),
//   h_t = a_t h_{t-1} + f_t i_t x_t;   a reset step has a = 0, f = 1 (a new
//   document starts there: nothing before it reaches it).
// Backward, reverse time on w_t = a_t d_t (what step t passes to step t-1):
//   d_t = dh_t + w_{t+1}  (w_T = dh_last),  dx = d f i,  dzi = d f x i (1-i),
//   dh/d(log a) = K = a h_{t-1} - i x a^2 / f  (0 on a reset step),
//   dzr = -lam d K r (1-r),  dlam = -sum d K r,  dbr = sum dzr,  dbi = sum dzi,
//   dh0 = w_0.
// The states (h0, h_last, dh_last, dh0, the step's pool) are fp32 whatever the
// storage type, so a sequence cut into pieces, or decoded step by step, carries
// no bf16 rounding from one piece to the next.  The backward pass takes
// h_{t-1} as the forward pass stored it (bf16 storage: rounded once, 2^-9), the
// way the other cells do: keeping fp32 states would double what it reads of h.
//
// The split.  An element costs about 54 instructions forward (49 without resets)
// and 75 backward (two gates, a decay, a square root), so at 8 to 32 bytes an
// element the issue slots are as scarce as the bytes, and the carry must not make
// an element's gates be computed twice.  The time axis is cut into S spans; a CTA
// owns one span of one channel strip and walks it through time, tile by tile, its
// state in shared memory, so CTAs wait for nothing but their own loads.  Wide
// problems have strips enough: S = 1 and one launch.  Narrow ones first run
// k_glr_agg, which computes only the spans' aggregates (A, B) -- backward that takes
// the decay and dh, two of the five inputs -- with every warp folding a run of its
// own and no barrier but the last; each CTA of k_glr_span then folds the aggregates
// of the spans before its own.  Every association depends on the shape alone: the
// same bits every run.
//
// Measured (HBM copy 6.78 TB/s).  Forward bf16 8192 x 16 x 4096 with resets: 1019 us,
// 4.2 TB/s, issue slots 75% busy (what warps wait for besides a slot: fixed latencies,
// loads, the pipes of the exponentials and roots).  Backward bf16 65536 x 1 x 1024 with
// resets, 128 spans: 289 us = k_glr_agg 84 + k_glr_span 196 (5.3 TB/s of what it moves)
// + the parameter sums 7; fp32 2048 x 32 x 1024: 381 us, 5.6 TB/s.  On the scan's engine, tiles carried from CTA
// to CTA, the same three took 1523, 667 and 391.
#include "lr_act.cuh"
#include "lr_launch.h"
#include "lr_tma.cuh"

#include <string.h>

#include <algorithm>
#include <type_traits>

namespace lrs {

namespace {

// A problem's tiles: L = NW R rows by 32 VEC channels; S spans of cps chunks.
struct SpanGeom {
    Geom g;         // T, C, D, n_chunks, n_ct and c / D
    uint32_t cps;   // chunks per span
    uint32_t S;
    int64_t nb;     // sequences (row pitch of reset)
    uint64_t wait_ns;   // limit of a wait
    uint32_t stalled;   // test: no tile is loaded, so that every wait runs out
};

// A thread's place in a block of rows: VEC channels of R rows, consecutive in scan
// order (reverse: falling time).  An address is the block's (the same for the
// whole warp) plus a 32-bit offset that no block changes.
template <class Op, int BLOCK_ROWS>
struct Lane {
    using S = typename Op::S;
    int64_t c;           // first channel
    int64_t cd;          // c mod D
    uint32_t seq;        // c / D
    uint32_t first;      // the thread's first row within the block, in scan order
    uint32_t row0;       // its time row
    bool cok;
    uint32_t vo[Op::R];  // byte offset of each row within the block
    __device__ __forceinline__ Lane(const SpanGeom& sg, uint32_t j, int first_row) {
        const int lane = threadIdx.x & 31;
        c = (int64_t)j * (32 * Op::VEC) + lane * Op::VEC;
        seq = (uint32_t)chan_seq(sg.g, c);
        cd = c - (int64_t)seq * sg.g.D;
        cok = c < sg.g.C;
        first = (uint32_t)first_row;
        row0 = (uint32_t)(Op::REV ? BLOCK_ROWS - 1 - first_row : first_row);
#pragma unroll
        for (int r = 0; r < Op::R; ++r) vo[r] = (uint32_t)((row(r) * sg.g.C + c) * (int64_t)sizeof(S));
    }
    __device__ __forceinline__ int64_t row(int r) const { return Op::REV ? (int64_t)row0 - r : (int64_t)row0 + r; }
    // row r of an array whose block starts at `block`
    template <typename T>
    __device__ __forceinline__ T* at(T* block, int r) const {
        using B = typename std::conditional<std::is_const<T>::value, const char, char>::type;
        return reinterpret_cast<T*>(reinterpret_cast<B*>(block) + vo[r]);
    }
};
// A block of rows: its first time row, that row's element offset, and whether
// all its rows are inside.
struct Block {
    int64_t t, at;
    bool full;
};
// Row r of the block's thread is inside the problem.
template <class L>
__device__ __forceinline__ bool inside(const L& ln, const Block& bk, const SpanGeom& sg, int r) {
    return ln.cok && (bk.full || bk.t + ln.row(r) < sg.g.T);
}
// The reset flags of a block's rows in scan order, bit k.  Where the warp's channels are
// one sequence's (one: the usual case), lane k reads row k's and a vote tells all; else
// a thread reads those of its own rows and the others' bits are set (they may be resets).
template <class Op, int BLOCK_ROWS, class L>
__device__ __forceinline__ uint32_t resets(const GlrIn& in, const L& ln, const Block& bk, const SpanGeom& sg, bool one) {
    if (in.reset == nullptr) return 0u;
    const uint8_t* b = in.reset + bk.t * sg.nb;
    if (one) {
        const int k = (int)(threadIdx.x & 31);
        const uint32_t row = Op::REV ? BLOCK_ROWS - 1 - k : k;
        bool hit = false;
        if (k < BLOCK_ROWS && (bk.full || bk.t + row < sg.g.T)) hit = __ldg(b + row * (uint32_t)sg.nb + ln.seq) != 0;
        return __ballot_sync(0xffffffffu, hit);
    }
    constexpr uint32_t own = (1u << Op::R) - 1, all = (1u << BLOCK_ROWS) - 1;
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < Op::R; ++r) {
        const uint32_t o = (uint32_t)ln.row(r) * (uint32_t)sg.nb + ln.seq;
        if (inside(ln, bk, sg, r) && __ldg(b + o) != 0) m |= 1u << r;
    }
    return (all & ~(own << ln.first)) | m << ln.first;
}
template <int R, class L>
__device__ __forceinline__ uint32_t own_resets(uint32_t m, const L& ln) {
    return m >> ln.first & ((1u << R) - 1);
}
// Whether the warp's channels all belong to its first lane's sequence.
template <class L>
__device__ __forceinline__ bool one_sequence(const L& ln) {
    const uint32_t first = __shfl_sync(0xffffffffu, ln.seq, 0);  // every lane takes part
    const bool same = ln.cok && ln.seq == first;
    return __all_sync(0xffffffffu, same) != 0;
}
// One row's VEC channels: from global memory (a block whose rows are all inside,
// h_{t-1}'s too, or any), or from the staged tile.
template <class Op, class L>
struct FromInside {
    const L& ln;
    int64_t at, C;
    template <typename S>
    __device__ __forceinline__ void ld(Pack<S, Op::VEC>& pk, int, const S* base, int r, int back = 0) const {
        pk.load(ln.at(base + at - back * C, r));
    }
};
template <class Op, class L>
struct FromGlobal {
    const L& ln;
    const Block& bk;
    const SpanGeom& sg;
    template <typename S>
    __device__ __forceinline__ void ld(Pack<S, Op::VEC>& pk, int, const S* base, int r, int back = 0) const {
        if (inside(ln, bk, sg, r) && bk.t + ln.row(r) >= back) pk.load(ln.at(base + bk.at - back * sg.g.C, r));
        else pk.ident(0.f);
    }
};
template <bool AGG, class Op, class L>
__device__ __forceinline__ void load_global(const typename Op::Params& p, const L& ln, const Block& bk, const SpanGeom& sg,
                                            typename Op::Regs& rg) {
    if (bk.full && ln.cok && bk.t > 0) Op::template load<AGG>(FromInside<Op, L>{ln, bk.at, sg.g.C}, p, rg);
    else Op::template load<AGG>(FromGlobal<Op, L>{ln, bk, sg}, p, rg);
}
template <class Op>
struct FromStage {  // rows and channels outside were filled with zeros
    const unsigned char* mine;  // the thread's first row in array 0
    template <typename S>
    __device__ __forceinline__ void ld(Pack<S, Op::VEC>& pk, int k, const S*, int r, int = 0) const {
        constexpr int pitch = 32 * Op::VEC * (int)sizeof(S);
        pk.load_shared(reinterpret_cast<const S*>(mine + tma_off<Op>(k) + (Op::REV ? -r : r) * pitch));
    }
};

// The per-feature constants of a lane: -lam / 16 and the biases times -log2 e;
// gen: a rate past the pairs' range (act_decay2), or 0, where the gradient of the
// decay is 0 by definition.
template <int VEC>
struct Feat {
    float l16[VEC], b2r[VEC], b2i[VEC];
    bool gen;
    __device__ __forceinline__ void load(const GlrIn& in, int64_t cd, bool cok) {
        float lam[VEC], br[VEC], bi[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) { lam[v] = 1.f; br[v] = bi[v] = 0.f; }
        if (cok) {
            load_feat(in.lam + cd, lam);
            load_feat(in.br + cd, br);
            load_feat(in.bi + cd, bi);
        }
        gen = false;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            gen = gen || !(lam[v] > 0.f && lam[v] <= kDecayMaxRate);
            l16[v] = -0.0625f * lam[v];
            b2r[v] = -kLog2e * br[v];
            b2i[v] = -kLog2e * bi[v];
        }
    }
    // both gates NaN: whatever the rows hold, the results are
    __device__ __forceinline__ void spoil() {
#pragma unroll
        for (int v = 0; v < VEC; ++v) b2r[v] = b2i[v] = __int_as_float(0x7fc00000);
    }
    // the general forms' arguments, exact up to the last bits of the products
    __device__ __forceinline__ float log_a(int v, float r) const { return 16.f * l16[v] * r; }
    __device__ __forceinline__ float gate(float z, float b2) const {
        return rcp_ftz(1.f + ex2_ftz(fmaf(z, -kLog2e, b2)));
    }
    __device__ static __forceinline__ void load_feat(const float* p, float (&x)[VEC]) {
        if constexpr (VEC == 2) {
            const float2 f = __ldg(reinterpret_cast<const float2*>(p));
            x[0] = f.x; x[1] = f.y;
        } else {
            x[0] = __ldg(p);
        }
    }
};

// A row's VEC values (bf16: one conversion for a pair).
template <typename S, int VEC>
__device__ __forceinline__ void store_row(S* p, const float (&x)[VEC]) {
    if constexpr (sizeof(S) == 2 && VEC == 2) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(x[1]), "f"(x[0]));
        asm volatile("st.global.cs.b32 [%0], %1;" ::"l"(p), "r"(w) : "memory");
    } else {
        store_vec<S, VEC>(p, x);
    }
}

// A reset step drops what is before it in scan order, finite or not (0 times an infinite
// or NaN state would be NaN).  Its decay is held as -0, which no other decay and no
// product of them is: where a decay underflows to +0, a NaN goes on through its document.
constexpr float kReset = -0.f;
__device__ __forceinline__ bool is_reset(float a) { return __float_as_uint(a) == 0x80000000u; }
__device__ __forceinline__ float scan_enter(float a, float s, float b) { return is_reset(a) ? b : __fmaf_rn(a, s, b); }
__device__ __forceinline__ void scan_join(float& A, float& B, float a, float b) {
    B = scan_enter(a, B, b);
    A = is_reset(a) ? kReset : A * a;  // -0 times a decay is -0
}
// An aggregate taken onto a state: of a block without resets, and with them.
struct ScanPlain {
    __device__ __forceinline__ float operator()(float a, float s, float b) const { return __fmaf_rn(a, s, b); }
};
struct ScanReset {
    __device__ __forceinline__ float operator()(float a, float s, float b) const { return scan_enter(a, s, b); }
};

// ------------------------------------------------------------------ forward

template <typename S>
struct GlrFwdParams {
    GlrIn in;
    const float* h0;
    S* h;
    float* h_last;
};

template <typename S_, int VEC_>
struct GlrFwdOp {
    using S = S_;
    static constexpr int VEC = VEC_, NW = 4, R = 4, MINB = 7;
    static constexpr bool REV = false;
    static constexpr int NSUM = 0;
    static constexpr float kMaxShared = 8.5e37f;  // just below 2^126
    using Params = GlrFwdParams<S>;
    struct Regs {
        Pack<S, VEC> x[R], zr[R], zi[R];
        uint32_t rs;  // reset rows of the block
    };
    struct Work {
        float fa[R][VEC], fb[R][VEC];  // scan element (a, f i x); a reset step: (kReset, i x)
    };
    __device__ static const float* init_ptr(const Params& p) { return p.h0; }

    static constexpr int TMA_N = 3;  // staged: x, zr, zi
    __host__ __device__ static constexpr int tma_shift(int) { return 0; }
    __host__ __device__ static constexpr int tma_extra(int) { return 0; }
    static void tma_arrays(const Params& p, const void** ptr) {
        ptr[0] = p.in.x;
        ptr[1] = p.in.zr;
        ptr[2] = p.in.zi;
    }

    template <bool AGG, class Src>
    __device__ static __forceinline__ void load(const Src& src, const Params& p, Regs& rg) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            src.ld(rg.x[r], 0, (const S*)p.in.x, r);
            src.ld(rg.zr[r], 1, (const S*)p.in.zr, r);
            src.ld(rg.zi[r], 2, (const S*)p.in.zi, r);
        }
    }
    // Two elements at a time (neighbouring channels, on the scalar path
    // neighbouring rows), one reciprocal for both gates: 1/(PQ) times Q and P.
    // Where PQ overflows, its reciprocal is flushed to 0 (from 2^126), or a rate is past
    // the pairs' range, the general forms.
    template <class L>
    __device__ static __forceinline__ void gates(const Params& p, const SpanGeom& sg, const L& ln, const Block& bk,
                                                 const Feat<VEC>& ft, const Regs& rg, Work& w,
                                                 float (&A)[VEC], float (&B)[VEC]) {
        static_assert(R * VEC % 2 == 0, "pairs");
        const f32x2 one = f2(1.f), nl = f2(-kLog2e);
        float pmax = 0.f;
#pragma unroll
        for (int e = 0; e < R * VEC; e += 2) {
            const int r0 = e / VEC, v0 = e % VEC, r1 = (e + 1) / VEC, v1 = (e + 1) % VEC;
            float a0, a1, b0, b1, t0, t1;
            f2_get(f2_fma(f2(rg.zr[r0].get(v0), rg.zr[r1].get(v1)), nl, f2(ft.b2r[v0], ft.b2r[v1])), a0, a1);
            f2_get(f2_fma(f2(rg.zi[r0].get(v0), rg.zi[r1].get(v1)), nl, f2(ft.b2i[v0], ft.b2i[v1])), b0, b1);
            const f32x2 P = f2_add(f2(ex2_ftz(a0), ex2_ftz(a1)), one);
            const f32x2 Q = f2_add(f2(ex2_ftz(b0), ex2_ftz(b1)), one);
            f2_get(f2_mul(P, Q), t0, t1);
            pmax = fmaxf(pmax, fmaxf(t0, t1));
            const f32x2 t = f2(rcp_ftz(t0), rcp_ftz(t1));
            const f32x2 u = f2_mul(f2_mul(t, P), f2(rg.x[r0].get(v0), rg.x[r1].get(v1)));
            float q0, q1;
            f32x2 a, q;
            act_decay2(f2_mul(f2_mul(t, Q), f2(ft.l16[v0], ft.l16[v1])), a, q);
            f2_get(q, q0, q1);
            f2_get(a, w.fa[r0][v0], w.fa[r1][v1]);
            f2_get(f2_mul(u, f2_mul(q, f2(rsqrt_ftz(q0), rsqrt_ftz(q1)))), w.fb[r0][v0], w.fb[r1][v1]);
        }
        const bool gen = ft.gen || pmax > kMaxShared;
#pragma unroll
        for (int v = 0; v < VEC; ++v) { A[v] = w.fa[0][v]; B[v] = w.fb[0][v]; }
#pragma unroll
        for (int r = 1; r < R; ++r)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                B[v] = __fmaf_rn(w.fa[r][v], B[v], w.fb[r][v]);
                A[v] *= w.fa[r][v];
            }
        const uint32_t rs = own_resets<R>(rg.rs, ln);
        if (gen || rs != 0 || !ln.cok || !bk.full) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool ok = inside(ln, bk, sg, r), reset = (rs >> r & 1u) != 0;
                if (ok && !reset && !gen) continue;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float a, q;
                    act_decay(ft.log_a(v, ft.gate(rg.zr[r].get(v), ft.b2r[v])), a, q);
                    const float u = ft.gate(rg.zi[r].get(v), ft.b2i[v]) * rg.x[r].get(v);
                    w.fa[r][v] = ok ? (reset ? kReset : a) : 1.f;
                    w.fb[r][v] = ok ? (reset ? u : sqrt_ftz(q) * u) : 0.f;
                }
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                A[v] = 1.f;
                B[v] = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) scan_join(A[v], B[v], w.fa[r][v], w.fb[r][v]);
            }
        }
    }
    // enter(s, e): s becomes the state entering the rows, each aggregate taken by e
    template <class L, class Enter>
    __device__ static __forceinline__ void finish(const Params& p, const SpanGeom& sg, const L& ln, const Block& bk,
                                                  const Feat<VEC>&, const Regs& rg, const Work& w,
                                                  float (&s)[VEC], float (&)[1][VEC], const Enter& enter) {
        S* h = p.h + bk.at;
        float o[R][VEC];
        if (rg.rs == 0) {
            enter(s, ScanPlain());
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[r][v] = s[v] = __fmaf_rn(w.fa[r][v], s[v], w.fb[r][v]);
        } else {
            enter(s, ScanReset());
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[r][v] = s[v] = scan_enter(w.fa[r][v], s[v], w.fb[r][v]);
        }
        if (bk.full) {
            if (ln.cok) {
#pragma unroll
                for (int r = 0; r < R; ++r) store_row(ln.at(h, r), o[r]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (inside(ln, bk, sg, r)) store_row(ln.at(h, r), o[r]);
        }
        if (bk.t + NW * R >= sg.g.T && p.h_last != nullptr && inside(ln, bk, sg, 0) && bk.t + ln.row(R) >= sg.g.T)
            store_vec<float, VEC>(p.h_last + ln.c, s);  // rows past the end kept s
    }
    template <class L>
    __device__ static __forceinline__ void last(const Params&, const L&, const float (&)[VEC]) {}
    __device__ static float* sums(const Params&) { return nullptr; }
};

// ----------------------------------------------------------------- backward

template <typename S>
struct GlrBwdParams {
    GlrIn in;
    const float* h0;
    const S* h;
    const S* dh;
    const float* dh_last;
    S* dx;
    S* dzr;
    S* dzi;
    float* dh0;
    float* partials;  // [3][S][C]: rate, decay bias, input bias
};

template <typename S_, int VEC_>
struct GlrBwdOp {
    using S = S_;
    static constexpr int VEC = VEC_, NW = 4, R = 4, MINB = 5;
    static constexpr bool REV = true;
    static constexpr int NSUM = 3;
    using Params = GlrBwdParams<S>;
    struct Regs {
        Pack<S, VEC> x[R], zr[R], zi[R], dh[R], hp[R];
        uint32_t rs;  // reset rows of the block
    };
    struct Work {
        float F[R][VEC];   // a (kReset on a reset step, 1 outside)
        float rr[R][VEC];  // r
        float q[R][VEC];   // 1 - a^2
        bool gen;          // some row needs the general forms
    };
    __device__ static const float* init_ptr(const Params& p) { return p.dh_last; }  // w_T

    static constexpr int TMA_N = 5;  // staged: x, zr, zi, dh, h (rows t0-1 .. t0+L-2)
    __host__ __device__ static constexpr int tma_shift(int k) { return k == 4 ? -1 : 0; }
    __host__ __device__ static constexpr int tma_extra(int) { return 0; }
    static void tma_arrays(const Params& p, const void** ptr) {
        ptr[0] = p.in.x;
        ptr[1] = p.in.zr;
        ptr[2] = p.in.zi;
        ptr[3] = p.dh;
        ptr[4] = p.h;
    }

    // AGG: what the aggregate needs, zr and dh.
    template <bool AGG, class Src>
    __device__ static __forceinline__ void load(const Src& src, const Params& p, Regs& rg) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            src.ld(rg.zr[r], 1, (const S*)p.in.zr, r);
            src.ld(rg.dh[r], 3, p.dh, r);
            if constexpr (!AGG) {
                src.ld(rg.x[r], 0, (const S*)p.in.x, r);
                src.ld(rg.zi[r], 2, (const S*)p.in.zi, r);
                src.ld(rg.hp[r], 4, p.h, r, 1);  // h_{t-1}; h0 is fp32: finish() reads it
            }
        }
    }
    // The decay alone, and the scan's element (F, F dh): w = F (dh + w').
    template <class L>
    __device__ static __forceinline__ void gates(const Params& p, const SpanGeom& sg, const L& ln, const Block& bk,
                                                 const Feat<VEC>& ft, const Regs& rg, Work& w,
                                                 float (&A)[VEC], float (&B)[VEC]) {
        static_assert(R * VEC % 2 == 0, "pairs");
        const f32x2 one = f2(1.f), nl = f2(-kLog2e);
#pragma unroll
        for (int e = 0; e < R * VEC; e += 2) {
            const int r0 = e / VEC, v0 = e % VEC, r1 = (e + 1) / VEC, v1 = (e + 1) % VEC;
            float a0, a1, t0, t1;
            f2_get(f2_fma(f2(rg.zr[r0].get(v0), rg.zr[r1].get(v1)), nl, f2(ft.b2r[v0], ft.b2r[v1])), a0, a1);
            f2_get(f2_add(f2(ex2_ftz(a0), ex2_ftz(a1)), one), t0, t1);
            w.rr[r0][v0] = rcp_ftz(t0);
            w.rr[r1][v1] = rcp_ftz(t1);
            f32x2 a, q;
            act_decay2(f2_mul(f2(w.rr[r0][v0], w.rr[r1][v1]), f2(ft.l16[v0], ft.l16[v1])), a, q);
            f2_get(a, w.F[r0][v0], w.F[r1][v1]);
            f2_get(q, w.q[r0][v0], w.q[r1][v1]);
        }
        const uint32_t rs = own_resets<R>(rg.rs, ln);
        w.gen = ft.gen || rs != 0 || (p.h0 != nullptr && bk.t + ln.row(R - 1) == 0);
#pragma unroll
        for (int v = 0; v < VEC; ++v) { A[v] = w.F[0][v]; B[v] = w.F[0][v] * rg.dh[0].get(v); }
#pragma unroll
        for (int r = 1; r < R; ++r)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                B[v] = w.F[r][v] * (rg.dh[r].get(v) + B[v]);
                A[v] *= w.F[r][v];
            }
        if (ft.gen || rs != 0 || !ln.cok || !bk.full) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool ok = inside(ln, bk, sg, r), reset = (rs >> r & 1u) != 0;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float a = w.F[r][v], q;
                    if (ft.gen) act_decay(ft.log_a(v, w.rr[r][v]), a, q);
                    w.F[r][v] = ok ? (reset ? kReset : a) : 1.f;
                }
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                A[v] = 1.f;
                B[v] = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float F = w.F[r][v];
                    B[v] = is_reset(F) ? 0.f : F * (rg.dh[r].get(v) + B[v]);
                    A[v] = is_reset(F) ? kReset : A[v] * F;
                }
            }
        }
    }
    template <class L, class Enter>
    __device__ static __forceinline__ void finish(const Params& p, const SpanGeom& sg, const L& ln, const Block& bk,
                                                  const Feat<VEC>& ft, const Regs& rg, const Work& w,
                                                  float (&s)[VEC], float (&sum)[3][VEC], const Enter& enter) {
        float d[R][VEC];  // d_t
        if (rg.rs == 0) {
            enter(s, ScanPlain());
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    d[r][v] = rg.dh[r].get(v) + s[v];
                    s[v] = w.F[r][v] * d[r][v];
                }
        } else {
            enter(s, ScanReset());
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    d[r][v] = rg.dh[r].get(v) + s[v];
                    s[v] = is_reset(w.F[r][v]) ? 0.f : w.F[r][v] * d[r][v];
                }
        }
        float dx[R][VEC], dzr[R][VEC], dzi[R][VEC], dl_[R][VEC];
        if (!w.gen) {
            const f32x2 one = f2(1.f), none = f2(-1.f), nl = f2(-kLog2e);
#pragma unroll
            for (int e = 0; e < R * VEC; e += 2) {
                const int r0 = e / VEC, v0 = e % VEC, r1 = (e + 1) / VEC, v1 = (e + 1) % VEC;
                float b0, b1, t0, t1;
                f2_get(f2_fma(f2(rg.zi[r0].get(v0), rg.zi[r1].get(v1)), nl, f2(ft.b2i[v0], ft.b2i[v1])), b0, b1);
                f2_get(f2_add(f2(ex2_ftz(b0), ex2_ftz(b1)), one), t0, t1);
                const f32x2 ii = f2(rcp_ftz(t0), rcp_ftz(t1));
                const f32x2 a = f2(w.F[r0][v0], w.F[r1][v1]);
                const f32x2 rf = f2(rsqrt_ftz(w.q[r0][v0]), rsqrt_ftz(w.q[r1][v1]));  // 1/f
                const f32x2 f = f2_mul(f2(w.q[r0][v0], w.q[r1][v1]), rf);
                const f32x2 u = f2_mul(ii, f2(rg.x[r0].get(v0), rg.x[r1].get(v1)));
                const f32x2 dd = f2(d[r0][v0], d[r1][v1]);
                const f32x2 df = f2_mul(dd, f);
                f2_get(f2_mul(df, ii), dx[r0][v0], dx[r1][v1]);
                f2_get(f2_mul(f2_mul(df, u), f2_fma(ii, none, one)), dzi[r0][v0], dzi[r1][v1]);
                // K = a (h - u a / f);  -d K r is lam's term, times lam (1 - r) zr's
                const f32x2 nh = f2_mul(f2(rg.hp[r0].get(v0), rg.hp[r1].get(v1)), none);
                const f32x2 nK = f2_mul(a, f2_fma(f2_mul(u, a), rf, nh));
                const f32x2 rr = f2(w.rr[r0][v0], w.rr[r1][v1]);
                const f32x2 dl = f2_mul(f2_mul(dd, nK), rr);
                // l16 = -lam / 16: -16 l16 dl (1 - r), the 16 exact
                const f32x2 lr = f2_mul(f2(ft.l16[v0], ft.l16[v1]), f2_fma(rr, f2(16.f), f2(-16.f)));
                f2_get(f2_mul(dl, lr), dzr[r0][v0], dzr[r1][v1]);
                f2_get(dl, dl_[r0][v0], dl_[r1][v1]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool reset = (own_resets<R>(rg.rs, ln) >> r & 1u) != 0;
                float hp[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) hp[v] = rg.hp[r].get(v);
                if (p.h0 != nullptr && ln.cok && bk.t + ln.row(r) == 0) load_vec<float, VEC>(p.h0 + ln.c, hp);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float rr = w.rr[r][v];
                    const float ii = ft.gate(rg.zi[r].get(v), ft.b2i[v]);
                    float a, q;
                    act_decay(ft.log_a(v, rr), a, q);
                    // where the decay is 1 to the last bit (q = 0) its gradient is
                    // 0: K's pole is cancelled by r (1-r) -> 0
                    const float rf = q > 0.f ? rsqrt_ftz(q) : q;
                    const float f = reset ? 1.f : q * rf;
                    const float u = ii * rg.x[r].get(v);
                    const float K = reset || q == 0.f ? 0.f : a * (hp[v] - u * a * rf);
                    const float dl = reset ? 0.f : -d[r][v] * K * rr;
                    dx[r][v] = d[r][v] * f * ii;
                    dzi[r][v] = d[r][v] * f * u * (1.f - ii);
                    dzr[r][v] = reset ? 0.f : dl * (-16.f * ft.l16[v]) * (1.f - rr);
                    dl_[r][v] = dl;
                }
            }
        }
        S *ox = p.dx + bk.at, *or_ = p.dzr + bk.at, *oi = p.dzi + bk.at;
        auto put = [&](int r) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                sum[0][v] += dl_[r][v];
                sum[1][v] += dzr[r][v];
                sum[2][v] += dzi[r][v];
            }
            store_row(ln.at(ox, r), dx[r]);
            store_row(ln.at(or_, r), dzr[r]);
            store_row(ln.at(oi, r), dzi[r]);
        };
        if (bk.full) {
            if (ln.cok) {
#pragma unroll
                for (int r = 0; r < R; ++r) put(r);
            }
        } else {  // rows outside hold a neighbour's d
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (inside(ln, bk, sg, r)) put(r);
        }
    }
    // the state after the last row of the scan: w_0
    template <class L>
    __device__ static __forceinline__ void last(const Params& p, const L& ln, const float (&s)[VEC]) {
        if (p.dh0 != nullptr && ln.cok) store_vec<float, VEC>(p.dh0 + ln.c, s);
    }
    __device__ static float* sums(const Params& p) { return p.partials; }
};

// ------------------------------------------------------------------ kernels

template <int VEC, int NW>
struct SpanSmem {
    float a[2][NW][32][VEC];
    float b[2][NW][32][VEC];
    float carry[2][32][VEC];
};

// The state entering a warp's rows: the carried one, with the aggregates of the warps
// before taken onto it by `take`.
template <int VEC, int NW, int PAR>
struct Entering {
    const SpanSmem<VEC, NW>& sm;
    int warp, lane;
    template <class Take>
    __device__ __forceinline__ void operator()(float (&s)[VEC], const Take& take) const {
#pragma unroll
        for (int w = 0; w < NW - 1; ++w)
            if (w < warp) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) s[v] = take(sm.a[PAR][w][lane][v], s[v], sm.b[PAR][w][lane][v]);
            }
    }
};

// The aggregate of span sp, strip j: (A, B) of its rows in scan order.  Warp w
// folds the span's row groups [w cps, (w+1) cps), loading one group ahead.
template <class Op>
__global__ void __launch_bounds__(Op::NW * 32)
    k_glr_agg(const typename Op::Params p, const SpanGeom sg, float2* __restrict__ agg) {
    constexpr int NW = Op::NW, VEC = Op::VEC;
    __shared__ float sa[NW][32][VEC], sb[NW][32][VEC];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sp = blockIdx.x / (uint32_t)sg.g.n_ct, j = blockIdx.x - sp * (uint32_t)sg.g.n_ct;
    // row groups of R: the warp's run, in scan order
    const int64_t g0 = ((int64_t)sp * NW + __shfl_sync(0xffffffffu, warp, 0)) * sg.cps;
    const int64_t rows = sg.g.n_chunks * (NW * Op::R);
    using L = Lane<Op, Op::R>;
    const L ln(sg, j, 0);
    auto place = [&](int64_t t) { return Block{t, t * sg.g.C, t + Op::R <= sg.g.T}; };
    const int64_t tstep = Op::REV ? -Op::R : Op::R, estep = tstep * sg.g.C;
    const bool one = one_sequence(ln);
    Feat<VEC> ft;
    ft.load(p.in, ln.cd, ln.cok);
    float A[VEC], B[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) { A[v] = 1.f; B[v] = 0.f; }
    typename Op::Regs rg[2];
    auto fetch = [&](const Block& bk, typename Op::Regs& r) {
        load_global<true, Op>(p, ln, bk, sg, r);
        r.rs = resets<Op, Op::R>(p.in, ln, bk, sg, one);
    };
    Block bk = place(Op::REV ? rows - Op::R - g0 * Op::R : g0 * Op::R);
    fetch(bk, rg[0]);
    for (uint32_t k = 0; k < sg.cps; k += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (k + h >= sg.cps) break;
            const int64_t t = bk.t + tstep;
            const Block nx{t, bk.at + estep, t + Op::R <= sg.g.T};
            if (k + h + 1 < sg.cps) fetch(nx, rg[h ^ 1]);
            typename Op::Work w;
            float a[VEC], b[VEC];
            Op::gates(p, sg, ln, bk, ft, rg[h], w, a, b);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {  // scan_join, told by the rows' flags
                B[v] = rg[h].rs != 0 ? b[v] : __fmaf_rn(a[v], B[v], b[v]);
                A[v] = rg[h].rs != 0 ? kReset : A[v] * a[v];
            }
            bk = nx;
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) { sa[warp][lane][v] = A[v]; sb[warp][lane][v] = B[v]; }
    __syncthreads();
    if (warp != 0 || !ln.cok) return;
#pragma unroll
    for (int w = 1; w < NW; ++w)
#pragma unroll
        for (int v = 0; v < VEC; ++v) scan_join(A[v], B[v], sa[w][lane][v], sb[w][lane][v]);
#pragma unroll
    for (int v = 0; v < VEC; ++v) agg[(int64_t)sp * sg.g.C + ln.c + v] = make_float2(A[v], B[v]);
}

// Thread 0: stage `it % ST` <- the tile of chunk q (scan order), strip j.
template <class Op, int ST>
__device__ __forceinline__ void span_issue(const SpanGeom& sg, const TmaDesc& td, unsigned char* ring, uint64_t* full,
                                           uint32_t it, uint32_t q, uint32_t j) {
    constexpr int L = Op::NW * Op::R, CW = 32 * Op::VEC;
    const int64_t tchunk = Op::REV ? sg.g.n_chunks - 1 - q : q;
    const int32_t x = (int32_t)(j * CW), y0 = (int32_t)(tchunk * L);
    const uint32_t st = it % ST;
    mbar_arrive_tx(&full[st], td.tx_bytes);
    unsigned char* dst = ring + st * tma_stage_bytes<Op>();
#pragma unroll
    for (int a = 0; a < Op::TMA_N; ++a)
        tma_load_2d(dst + tma_off<Op>(a), &td.map[a], x, y0 + Op::tma_shift(a), &full[st]);
}

// Span sp of strip j.  ST > 0: tiles through a ring of ST stages filled by TMA;
// ST = 0 (rows TMA cannot take): through registers, one tile ahead.  One barrier
// per tile: the warps' aggregates alternate between two buffers, every warp folds
// those before its own onto the carried state, and the last one carries on.
template <class Op, int ST>
__global__ void __launch_bounds__(Op::NW * 32, ST > 0 ? Op::MINB : Op::MINB - 2)
    k_glr_span(const typename Op::Params p, const SpanGeom sg, const float2* __restrict__ agg, uint32_t* err,
               const __grid_constant__ TmaDesc td) {
    constexpr int NW = Op::NW, VEC = Op::VEC, L = NW * Op::R;
    constexpr int NS = Op::NSUM > 0 ? Op::NSUM : 1;
    extern __shared__ unsigned char dyn[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dyn) + 127) & ~(uintptr_t)127);
    __shared__ SpanSmem<VEC, NW> sm;
    __shared__ __align__(8) uint64_t full[ST > 0 ? ST : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sp = blockIdx.x / (uint32_t)sg.g.n_ct, j = blockIdx.x - sp * (uint32_t)sg.g.n_ct;
    const uint32_t q0 = sp * sg.cps;
    const uint32_t n = (uint32_t)sg.g.n_chunks - q0 < sg.cps ? (uint32_t)sg.g.n_chunks - q0 : sg.cps;
    if (ST > 0 && threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(&full[i], 1);
        mbar_init_fence();
        for (uint32_t i = 0; i < (uint32_t)ST && i < n && !sg.stalled; ++i)
            span_issue<Op, ST>(sg, td, ring, full, i, q0 + i, j);
    }
    using Ln = Lane<Op, L>;
    const Ln ln(sg, j, warp * Op::R);
    const int64_t tstep = Op::REV ? -L : L, estep = tstep * sg.g.C;
    const bool one = one_sequence(ln);
    Block bk;
    bk.t = (Op::REV ? sg.g.n_chunks - 1 - q0 : (int64_t)q0) * L;
    bk.at = bk.t * sg.g.C;
    bk.full = bk.t + L <= sg.g.T;
    typename Op::Regs rg, ahead;
    if constexpr (ST == 0) load_global<false, Op>(p, ln, bk, sg, rg);
    rg.rs = resets<Op, L>(p.in, ln, bk, sg, one);
    Feat<VEC> ft;
    ft.load(p.in, ln.cd, ln.cok);
    const uint32_t mine = ln.row0 * (32 * VEC * (uint32_t)sizeof(typename Op::S)) + lane * (VEC * (uint32_t)sizeof(typename Op::S));
    {  // the state entering the span: each warp folds its share of the spans before
        float A[VEC], B[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) { A[v] = 1.f; B[v] = 0.f; }
        const uint32_t lo = (uint32_t)((uint64_t)sp * warp / NW), hi = (uint32_t)((uint64_t)sp * (warp + 1) / NW);
        if (ln.cok) {
#pragma unroll 4
            for (uint32_t k = lo; k < hi; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float2 e = agg[(int64_t)k * sg.g.C + ln.c + v];
                    scan_join(A[v], B[v], e.x, e.y);
                }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) { sm.a[1][warp][lane][v] = A[v]; sm.b[1][warp][lane][v] = B[v]; }
        __syncthreads();
        if (warp == 0) {
            float s[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) s[v] = 0.f;
            const float* ip = Op::init_ptr(p);
            if (ip != nullptr && ln.cok) load_vec<float, VEC>(ip + ln.c, s);
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
                for (int v = 0; v < VEC; ++v) s[v] = scan_enter(sm.a[1][w][lane][v], s[v], sm.b[1][w][lane][v]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) sm.carry[0][lane][v] = s[v];
        }
        // carry[0] is read after the first tile's barrier
    }
    float sum[NS][VEC];
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int v = 0; v < VEC; ++v) sum[k][v] = 0.f;
    bool dead = false;
    // one tile; PAR: its buffer (and stage: two), known to the compiler
    auto tile = [&](auto par_, uint32_t it) {
        constexpr int PAR = decltype(par_)::value;
        const bool more = it + 1 < n;
        const int64_t t = bk.t + tstep;
        const Block nx{t, bk.at + estep, t + L <= sg.g.T};
        if constexpr (ST > 0) {
            if (!mbar_wait(&full[PAR], (it >> 1) & 1u, err, sg.wait_ns)) {
                dead = true;  // this tile's results and the next ones' become NaN
                atomicOr(err, ERRBIT_TIMEOUT);
                ft.spoil();
            }
            Op::template load<false>(FromStage<Op>{ring + PAR * tma_stage_bytes<Op>() + mine}, p, rg);
        } else if (more) {
            load_global<false, Op>(p, ln, nx, sg, ahead);
        }
        if (more) ahead.rs = resets<Op, L>(p.in, ln, nx, sg, one);
        float A[VEC], B[VEC];
        typename Op::Work w;
        Op::gates(p, sg, ln, bk, ft, rg, w, A, B);
#pragma unroll
        for (int v = 0; v < VEC; ++v) { sm.a[PAR][warp][lane][v] = A[v]; sm.b[PAR][warp][lane][v] = B[v]; }
        csync<NW>();  // the tile's one barrier: its stage has been read too
        if (ST > 0 && threadIdx.x == 0 && it + ST < n && !dead)
            span_issue<Op, ST>(sg, td, ring, full, it + ST, q0 + it + ST, j);
        float s[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[v] = sm.carry[PAR][lane][v];
        Op::finish(p, sg, ln, bk, ft, rg, w, s, sum, Entering<VEC, NW, PAR>{sm, warp, lane});
        if (warp == NW - 1) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) sm.carry[PAR ^ 1][lane][v] = s[v];
            if (!more && sp + 1 == sg.S) Op::last(p, ln, s);
        }
        if constexpr (ST == 0) rg = ahead;
        else rg.rs = ahead.rs;
        bk = nx;
    };
    static_assert(ST == 0 || ST == 2, "a stage per buffer");
    for (uint32_t it = 0; it < n; it += 2) {
        tile(std::integral_constant<int, 0>{}, it);
        if (it + 1 < n) tile(std::integral_constant<int, 1>{}, it + 1);
    }
    if (ST > 0 && dead && threadIdx.x == 0) {  // copies still in flight land first
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(10000);
    }
    if constexpr (Op::NSUM > 0) {  // parameter sums of the span, the warps' in order
        __syncthreads();
        float(*ps)[32][VEC] = &sm.a[0][0];
#pragma unroll
        for (int k = 0; k < Op::NSUM; ++k) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) ps[warp][lane][v] = sum[k][v];
            __syncthreads();
            if (warp == 0 && ln.cok) {
                float* out = Op::sums(p) + ((int64_t)k * sg.S + sp) * sg.g.C + ln.c;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float t = ps[0][lane][v];
#pragma unroll
                    for (int w2 = 1; w2 < NW; ++w2) t += ps[w2][lane][v];
                    out[v] = t;
                }
            }
            __syncthreads();
        }
    }
}

// One step of every row: four inputs and the state of the row's slot, each
// element once.  A row is a few thousand elements at most and the rows few, so
// the launch and one round trip to memory are the time.  A slot past the pool
// is treated as padding and recorded in the error word.
template <typename S, int VEC>
__global__ void __launch_bounds__(256)
    k_glr_step(const S* __restrict__ x, const S* __restrict__ zr, const S* __restrict__ zi,
               const float* __restrict__ lam, const float* __restrict__ br,
               const float* __restrict__ bi, const uint8_t* __restrict__ reset,
               const int32_t* __restrict__ slots, float* __restrict__ state, S* __restrict__ h,
               int64_t rows, int64_t n_slots, int64_t D, uint32_t* err) {
    const int64_t d = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (d >= D) return;
    float vl[VEC], vr[VEC], vi[VEC];
    load_param<VEC>(lam + d, vl);
    load_param<VEC>(br + d, vr);
    load_param<VEC>(bi + d, vi);
    for (int64_t b = blockIdx.y; b < rows; b += gridDim.y) {
        const int64_t slot = slots != nullptr ? (int64_t)__ldg(slots + b) : b;
        Pack<S, VEC> px, pr, pi;
        px.load(x + b * D + d);
        pr.load(zr + b * D + d);
        pi.load(zi + b * D + d);
        const bool rs = reset != nullptr && __ldg(reset + b) != 0;
        float s[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[v] = 0.f;
        if (slot < 0 || slot >= n_slots) {
            if (slot >= n_slots) atomicOr(err, ERRBIT_INDEX);
            store_vec<S, VEC>(h + b * D + d, s);
            continue;
        }
        float* sp = state + slot * D + d;
        if constexpr (VEC == 4) {
            const float4 f4 = *reinterpret_cast<const float4*>(sp);
            s[0] = f4.x; s[1] = f4.y; s[2] = f4.z; s[3] = f4.w;
        } else {
            s[0] = *sp;
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float a, q;
            act_decay(-vl[v] * act_sigmoid(pr.get(v) + vr[v]), a, q);
            const float u = act_sigmoid(pi.get(v) + vi[v]) * px.get(v);
            s[v] = rs ? u : fmaf(a, s[v], sqrt_ftz(q) * u);
        }
        if constexpr (VEC == 4) *reinterpret_cast<float4*>(sp) = make_float4(s[0], s[1], s[2], s[3]);
        else *sp = s[0];
        store_vec<S, VEC>(h + b * D + d, s);
    }
}


// --------------------------------------------------------------------- host

constexpr int kSpanStages = 2;

template <class Op, int ST>
cudaError_t span_slots(int* slots) {  // CTAs resident on the GPU
    static int known[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    int& n = known[dev & 63];
    constexpr size_t smem = ST > 0 ? (size_t)ST * tma_stage_bytes<Op>() + 128 : 0;
    if (n <= 0) {
        if (ST > 0) {
            cudaError_t e = cudaFuncSetAttribute(k_glr_span<Op, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            e = cudaFuncSetAttribute(k_glr_span<Op, ST>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     (int)cudaSharedmemCarveoutMaxShared);
            if (e != cudaSuccess) return e;
        }
        int b = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, k_glr_span<Op, ST>, Op::NW * 32, smem) != cudaSuccess || b < 1)
            b = 1;
        n = b * sm_count();
    }
    *slots = n;
    return cudaSuccess;
}

template <class Op, int ST>
cudaError_t span_run(const typename Op::Params& p, const GlrSpans& pl, const Geom& g, float2* agg, uint32_t* err,
                     cudaStream_t s) {
    int slots = 0;
    const cudaError_t e = span_slots<Op, ST>(&slots);
    if (e != cudaSuccess) return e;
    const SpanGeom sg{g, (uint32_t)pl.cps, (uint32_t)pl.S, g.C / g.D, pl.stall_ns ? pl.stall_ns : kMbarLimitNs, pl.stall_ns != 0};
    TmaDesc td;
    memset(&td, 0, sizeof td);
    if (ST > 0) {
        const void* ptr[TMA_MAX_ARR] = {};
        Op::tma_arrays(p, ptr);
        for (int a = 0; a < Op::TMA_N; ++a) {
            if (!tma_encode(&td.map[a], ptr[a], sizeof(typename Op::S) == 2 ? 1 : 0, g.T, g.C, 32 * Op::VEC, Op::NW * Op::R))
                return cudaErrorInvalidValue;
            td.tx_bytes += tma_arr_bytes<Op>(a);
        }
    }
    if (pl.S > 1) {
        k_glr_agg<Op><<<(unsigned)((pl.S - 1) * g.n_ct), Op::NW * 32, 0, s>>>(p, sg, agg);
        const cudaError_t e2 = cudaGetLastError();
        if (e2 != cudaSuccess) return e2;
    }
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof lc);
    lc.gridDim = dim3((unsigned)(pl.S * g.n_ct));
    lc.blockDim = dim3(Op::NW * 32);
    lc.dynamicSmemBytes = ST > 0 ? (size_t)ST * tma_stage_bytes<Op>() + 128 : 0;
    lc.stream = s;
    return cudaLaunchKernelEx(&lc, k_glr_span<Op, ST>, p, sg, (const float2*)agg, err, td);
}

template <template <typename, int> class Op, class Make>
cudaError_t span_dispatch(int dtype, const GlrSpans& pl, const Geom& g, float2* agg, uint32_t* err, cudaStream_t s,
                          const Make& make) {
    if (dtype == 0) {
        const auto p = make((float*)nullptr);
        if (pl.tma) return span_run<Op<float, 2>, kSpanStages>(p, pl, g, agg, err, s);
        return pl.vec ? span_run<Op<float, 2>, 0>(p, pl, g, agg, err, s) : span_run<Op<float, 1>, 0>(p, pl, g, agg, err, s);
    }
    const auto p = make((__nv_bfloat16*)nullptr);
    if (pl.tma) return span_run<Op<__nv_bfloat16, 2>, kSpanStages>(p, pl, g, agg, err, s);
    return pl.vec ? span_run<Op<__nv_bfloat16, 2>, 0>(p, pl, g, agg, err, s)
                  : span_run<Op<__nv_bfloat16, 1>, 0>(p, pl, g, agg, err, s);
}

Geom span_geom(const GlrSpans& pl, int64_t T, int64_t C, int64_t D) {
    Geom g{};
    g.T = T;
    g.C = C;
    g.D = D;
    set_channel_div(g);
    g.n_chunks = pl.n_chunks;
    g.n_ct = (int)pl.n_ct;
    return g;
}

}  // namespace

// The spans of a problem.  vec: the 16-byte path's pointers and D a multiple of 4.
//
// One span while the strips alone keep the SMs busy, else the aggregates' pass,
// which reads some inputs again, costs less than idle slots do.  Measured with
// 2^27 elements, one span against the spans chosen here, us:
//   strips        128        192        256        320        384
//   bf16 fwd   666 / 432  526 / 427  396 / 424  358 / 417  302 / 418
//   fp32 fwd   690 / 547  529 / 541  418 / 538  392 / 531  351 / 536
//   bf16 bwd   884 / 482  687 / 482  524 / 474  527 / 478  450 / 474
//   fp32 bwd   930 / 808  769 / 805  656 / 805  681 / 796  705 / 814
// Cut: at first as many spans as make one CTA for every slot (7 an SM forward, 5
// backward); where spans stay 32 tiles long, up to three times as many, which even
// out the SMs (4096 channels of 32768 steps, when it was chosen: bf16 451 -> 429 us
// forward, 532 -> 486 backward, fp32 902 -> 814; of 2048 steps, where a span would be
// three tiles, 35 -> 39 forward, so not there).  At least two tiles a span.
GlrSpans glr_spans(bool bwd, int dtype, bool vec, int64_t T, int64_t C) {
    GlrSpans p{};
    const int es = dtype == 1 ? 2 : 4;
    p.rows = 16;
    p.vec = vec;
    p.tma = vec && (C * es) % 16 == 0 && C >= 64 && T < ((int64_t)1 << 30) && C < ((int64_t)1 << 30);
    const int64_t cw = vec ? 64 : 32;
    p.n_chunks = (T + p.rows - 1) / p.rows;
    p.n_ct = (C + cw - 1) / cw;
    const int64_t slots = (bwd ? 5 : 7) * (int64_t)kSpanSms;
    // strips an SM, in quarters, from which one span is faster
    const int64_t enough = dtype == 1 ? (bwd ? 9 : 6) : (bwd ? 4 : 5);
    p.S = 1;
    if (4 * p.n_ct < enough * kSpanSms) {
        p.S = std::max(slots / p.n_ct, std::min(3 * slots / p.n_ct, p.n_chunks / 32));
        p.S = std::max<int64_t>(std::min(p.S, p.n_chunks / 2), 1);
    }
    p.cps = (p.n_chunks + p.S - 1) / p.S;
    p.S = (p.n_chunks + p.cps - 1) / p.cps;
    return p;
}

cudaError_t launch_glr_fwd(int dtype, const GlrSpans& pl, const GlrIn& in, const float* h0, void* h, float* h_last,
                           float* scratch, int64_t T, int64_t C, int64_t D, uint32_t* err, cudaStream_t s) {
    const Geom g = span_geom(pl, T, C, D);
    auto make = [&](auto* tag) {
        using S = std::remove_pointer_t<decltype(tag)>;
        return GlrFwdParams<S>{in, h0, (S*)h, h_last};
    };
    return span_dispatch<GlrFwdOp>(dtype, pl, g, (float2*)scratch, err, s, make);
}

cudaError_t launch_glr_bwd(int dtype, const GlrSpans& pl, const GlrIn& in, const float* h0, const void* h, const void* dh,
                           const float* dh_last, void* dx, void* dzr, void* dzi, float* dh0, float* scratch, int64_t T,
                           int64_t C, int64_t D, uint32_t* err, cudaStream_t s) {
    const Geom g = span_geom(pl, T, C, D);
    float* partials = scratch + 2 * pl.S * C;
    auto make = [&](auto* tag) {
        using S = std::remove_pointer_t<decltype(tag)>;
        return GlrBwdParams<S>{in, h0, (const S*)h, (const S*)dh, dh_last, (S*)dx, (S*)dzr, (S*)dzi, dh0, partials};
    };
    return span_dispatch<GlrBwdOp>(dtype, pl, g, (float2*)scratch, err, s, make);
}

template <typename S, int VEC>
static cudaError_t glr_step_t(const GlrIn& in, const int32_t* slots, float* state, void* h,
                              int64_t rows, int64_t n_slots, int64_t D, uint32_t* err,
                              cudaStream_t s) {
    const int64_t lanes = (D + VEC - 1) / VEC;
    const int threads = lanes >= 256 ? 256 : (int)((lanes + 31) / 32 * 32);
    const int64_t bx = (lanes + threads - 1) / threads;
    if (bx > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t by = rows < 65535 ? rows : 65535;
    k_glr_step<S, VEC><<<dim3((unsigned)bx, (unsigned)by), threads, 0, s>>>(
        (const S*)in.x, (const S*)in.zr, (const S*)in.zi, in.lam, in.br, in.bi, in.reset, slots, state,
        (S*)h, rows, n_slots, D, err);
    return cudaGetLastError();
}

cudaError_t launch_glr_step(int dtype, bool vec, const GlrIn& in, const int32_t* slots, float* state,
                            void* h, int64_t rows, int64_t n_slots, int64_t D, uint32_t* err,
                            cudaStream_t s) {
    if (dtype == 0)
        return vec ? glr_step_t<float, 4>(in, slots, state, h, rows, n_slots, D, err, s)
                   : glr_step_t<float, 1>(in, slots, state, h, rows, n_slots, D, err, s);
    return vec ? glr_step_t<__nv_bfloat16, 4>(in, slots, state, h, rows, n_slots, D, err, s)
               : glr_step_t<__nv_bfloat16, 1>(in, slots, state, h, rows, n_slots, D, err, s);
}

}  // namespace lrs
