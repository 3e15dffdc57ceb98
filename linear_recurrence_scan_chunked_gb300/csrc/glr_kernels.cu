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
// Bytes bound it: 4 arrays forward, 8 backward, each element crossing HBM once.
#include "lr_act.cuh"
#include "lr_launch.h"
#include "lr_persist.cuh"

namespace lrs {

template <typename S>
struct GlrFwdParams {
    const S* x;
    const S* zr;
    const S* zi;
    const float* lam;
    const float* br;
    const float* bi;
    const uint8_t* reset;
    const float* h0;
    S* h;
    float* h_last;
    int64_t nb;  // sequences (row pitch of reset)
};

template <typename S_, int VEC_, int NW_, int R_>
struct GlrFwdOp {
    using S = S_;
    static constexpr bool STRIP_ONE_BARRIER = LR_STRIP_ONEB != 0;
    static constexpr int VEC = VEC_, NW = NW_, R = R_, MINB = 2;
    static constexpr bool REV = false;
    static constexpr int IN_ARRAYS = 3;  // x, zr, zi
    static constexpr bool SCRATCH_IN_CARRY = false;
    using Params = GlrFwdParams<S>;
    struct Regs {
        Pack<S, VEC> x[R], zr[R], zi[R];
        uint8_t rs[R];
    };
    struct Work {
        float fa[R][VEC], fb[R][VEC];  // scan element (a, f i x)
    };
    struct Smem {
        int unused;
    };
    struct Acc {};
    __device__ static void acc_init(Acc&) {}
    __device__ static bool skip(const Params&) { return false; }
    __host__ __device__ static const float* init_ptr(const Params& p) { return p.h0; }

    static constexpr int TMA_N = 3;  // staged: x, zr, zi
    __host__ __device__ static constexpr int tma_shift(int) { return 0; }
    __host__ __device__ static constexpr int tma_extra(int) { return 0; }
    static void tma_arrays(const Params& p, const void** ptr) {
        ptr[0] = p.x;
        ptr[1] = p.zr;
        ptr[2] = p.zi;
    }

    template <class Src>
    __device__ static void load(const Src& src, const Params& p, const Geom& g,
                                const TileCoord& tc, Regs& rg) {
        // a lane's channels belong to one sequence (VEC divides D)
        const uint8_t* rs = p.reset != nullptr && tc.cok ? p.reset + chan_seq(g, tc.c) : nullptr;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t t = tc.t0 + r;
            rg.rs[r] = 0;
            if (tc.cok && t < g.T) {
                src.ld(rg.x[r], 0, p.x, t);
                src.ld(rg.zr[r], 1, p.zr, t);
                src.ld(rg.zi[r], 2, p.zi, t);
                if (rs != nullptr) rg.rs[r] = __ldg(rs + t * p.nb);
            } else {
                rg.x[r].ident(0.f);
                rg.zr[r].ident(0.f);
                rg.zi[r].ident(0.f);
            }
        }
    }
    // Two elements at a time (neighbouring channels on the vector path,
    // neighbouring rows on the scalar one), one reciprocal for both gates:
    // 1/(AB) times B and A.  Gates shut past 2^-60 and decays past e^-2 take the
    // general forms.
    __device__ static void aggregate(const Params& p, const Geom& g, const TileCoord& tc,
                                     const Regs& rg, Work& w, float (&A)[VEC], float (&B)[VEC],
                                     bool) {
        static_assert(R * VEC % 2 == 0, "pairs");
        float lam[VEC], br[VEC], bi[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) { lam[v] = br[v] = bi[v] = 0.f; A[v] = 1.f; B[v] = 0.f; }
        if (tc.cok) {
            load_param<VEC>(p.lam + tc.cd, lam);
            load_param<VEC>(p.br + tc.cd, br);
            load_param<VEC>(p.bi + tc.cd, bi);
        }
        float l8[VEC], b2r[VEC], b2i[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            l8[v] = -0.125f * lam[v];
            b2r[v] = -kLog2e * br[v];
            b2i[v] = -kLog2e * bi[v];
        }
        const f32x2 one = f2(1.f), nl = f2(-kLog2e);
        float emax = 0.f, xmin = 0.f;
#pragma unroll
        for (int e = 0; e < R * VEC; e += 2) {
            const int r0 = e / VEC, v0 = e % VEC, r1 = (e + 1) / VEC, v1 = (e + 1) % VEC;
            float er0, er1, ei0, ei1;
            f2_get(f2_fma(f2(rg.zr[r0].get(v0), rg.zr[r1].get(v1)), nl, f2(b2r[v0], b2r[v1])), er0, er1);
            f2_get(f2_fma(f2(rg.zi[r0].get(v0), rg.zi[r1].get(v1)), nl, f2(b2i[v0], b2i[v1])), ei0, ei1);
            emax = fmaxf(fmaxf(emax, fmaxf(er0, er1)), fmaxf(ei0, ei1));
            const f32x2 P = f2_add(f2(ex2_ftz(er0), ex2_ftz(er1)), one);
            const f32x2 Q = f2_add(f2(ex2_ftz(ei0), ex2_ftz(ei1)), one);
            float t0, t1;
            f2_get(f2_mul(P, Q), t0, t1);
            const f32x2 t = f2(rcp_ftz(t0), rcp_ftz(t1));
            const f32x2 x = f2_mul(f2_mul(t, Q), f2(l8[v0], l8[v1]));
            const f32x2 u = f2_mul(f2_mul(t, P), f2(rg.x[r0].get(v0), rg.x[r1].get(v1)));
            float x0, x1, q0, q1;
            f2_get(x, x0, x1);
            xmin = fminf(xmin, fminf(x0, x1));
            f32x2 a, nq;
            act_decay2(x, a, nq);
            f2_get(nq, q0, q1);
            f2_get(a, w.fa[r0][v0], w.fa[r1][v1]);
            f2_get(f2_mul(u, f2(sqrt_ftz(-q0), sqrt_ftz(-q1))), w.fb[r0][v0], w.fb[r1][v1]);
        }
        bool any = emax > kGateMaxExp || xmin < kDecayMinX || !(tc.cok && tc.t0 + R - 1 < g.T);
#pragma unroll
        for (int r = 0; r < R; ++r) any = any || rg.rs[r] != 0;
        if (any) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool ok = tc.cok && tc.t0 + r < g.T, reset = rg.rs[r] != 0;
                if (ok && !reset && !(emax > kGateMaxExp || xmin < kDecayMinX)) continue;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float a, q;
                    act_decay(-lam[v] * act_sigmoid(rg.zr[r].get(v) + br[v]), a, q);
                    const float u = act_sigmoid(rg.zi[r].get(v) + bi[v]) * rg.x[r].get(v);
                    w.fa[r][v] = ok ? (reset ? 0.f : a) : 1.f;
                    w.fb[r][v] = ok ? (reset ? u : sqrt_ftz(q) * u) : 0.f;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                B[v] = __fmaf_rn(w.fa[r][v], B[v], w.fb[r][v]);
                A[v] *= w.fa[r][v];
            }
    }
    __device__ static void finish(const Params& p, const Geom& g, const TileCoord& tc,
                                  const Regs&, Work& w, float (&s)[VEC], Smem&, Acc&) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t t = tc.t0 + r;
#pragma unroll
            for (int v = 0; v < VEC; ++v) s[v] = w.fa[r][v] * s[v] + w.fb[r][v];
            if (tc.cok && t < g.T) {
                store_vec<S, VEC>(p.h + t * g.C + tc.c, s);
                if (t == g.T - 1 && p.h_last != nullptr) store_vec<float, VEC>(p.h_last + tc.c, s);
            }
        }
    }
    __device__ static void at_exit(const Params&, Smem&, Acc&) {}
};

template <typename S>
struct GlrBwdParams {
    const S* x;
    const S* zr;
    const S* zi;
    const float* lam;
    const float* br;
    const float* bi;
    const uint8_t* reset;
    const float* h0;
    const S* h;
    const S* dh;
    const float* dh_last;
    S* dx;
    S* dzr;
    S* dzi;
    float* dh0;
    float* partials;  // [3][n_chunks][C]: rate, decay bias, input bias
    int64_t nb;
};

template <typename S_, int VEC_, int NW_, int R_>
struct GlrBwdOp {
    using S = S_;
    static constexpr int VEC = VEC_, NW = NW_, R = R_, MINB = 2;
    static constexpr bool REV = true;
    static constexpr int IN_ARRAYS = 5;  // x, zr, zi, dh, h_{t-1}
    using Params = GlrBwdParams<S>;
    struct Regs {
        Pack<S, VEC> x[R], zr[R], zi[R], dh[R], hp[R];
        uint8_t rs[R];
    };
    struct Work {
        float F[R][VEC];   // a
        float CX[R][VEC];  // dx / d = f i
        float CI[R][VEC];  // dzi / d = f x i (1-i)
        float KR[R][VEC];  // dlam's term / d = -K r
        float CR[R][VEC];  // dzr / d = -lam K r (1-r)
    };
    struct Smem {
        float ps[3][NW][32][VEC];
    };
    // 12 KB of their own: more than the carry's warp aggregates hold, and two
    // CTAs of 40 KB stages still fit an SM.
    static constexpr bool SCRATCH_IN_CARRY = false;
    struct Acc {
        float s[3][VEC];  // parameter sums over a run of tiles (acc_run)
    };
    __device__ static void acc_init(Acc& a) {
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) a.s[k][v] = 0.f;
    }
    __device__ static bool skip(const Params&) { return false; }
    __host__ __device__ static const float* init_ptr(const Params& p) { return p.dh_last; }  // w_T

    static constexpr int TMA_N = 5;  // staged: x, zr, zi, dh, h (rows t0-1 .. t0+L-2)
    __host__ __device__ static constexpr int tma_shift(int k) { return k == 4 ? -1 : 0; }
    __host__ __device__ static constexpr int tma_extra(int) { return 0; }
    static void tma_arrays(const Params& p, const void** ptr) {
        ptr[0] = p.x;
        ptr[1] = p.zr;
        ptr[2] = p.zi;
        ptr[3] = p.dh;
        ptr[4] = p.h;
    }

    template <class Src>
    __device__ static void load(const Src& src, const Params& p, const Geom& g,
                                const TileCoord& tc, Regs& rg) {
        const uint8_t* rs = p.reset != nullptr && tc.cok ? p.reset + chan_seq(g, tc.c) : nullptr;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t t = tc.t0 - r;
            rg.rs[r] = 0;
            if (tc.cok && t < g.T) {
                src.ld(rg.x[r], 0, p.x, t);
                src.ld(rg.zr[r], 1, p.zr, t);
                src.ld(rg.zi[r], 2, p.zi, t);
                src.ld(rg.dh[r], 3, p.dh, t);
                if (t > 0) src.ld(rg.hp[r], 4, p.h, t - 1);
                else rg.hp[r].ident(0.f);  // h0 is fp32: aggregate() reads it
                if (rs != nullptr) rg.rs[r] = __ldg(rs + t * p.nb);
            } else {
                rg.x[r].ident(0.f);
                rg.zr[r].ident(0.f);
                rg.zi[r].ident(0.f);
                rg.dh[r].ident(0.f);
                rg.hp[r].ident(0.f);
            }
        }
    }
    // As the forward pass, two elements at a time; a square root's pole (a decay
    // of 1 to the last bit) takes the general form too.  The pass that only wants
    // the aggregate (side = false) needs no more than the decay.
    __device__ static void aggregate(const Params& p, const Geom& g, const TileCoord& tc,
                                     const Regs& rg, Work& w, float (&A)[VEC], float (&B)[VEC],
                                     bool side) {
        static_assert(R * VEC % 2 == 0, "pairs");
        float lam[VEC], br[VEC], bi[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) { lam[v] = br[v] = bi[v] = 0.f; A[v] = 1.f; B[v] = 0.f; }
        if (tc.cok) {
            load_param<VEC>(p.lam + tc.cd, lam);
            load_param<VEC>(p.br + tc.cd, br);
            load_param<VEC>(p.bi + tc.cd, bi);
        }
        float l8[VEC], b2r[VEC], b2i[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            l8[v] = -0.125f * lam[v];
            b2r[v] = -kLog2e * br[v];
            b2i[v] = -kLog2e * bi[v];
        }
        const f32x2 one = f2(1.f), none = f2(-1.f), nl = f2(-kLog2e);
        float emax = 0.f, xmin = 0.f, qmin = 1.f;
#pragma unroll
        for (int e = 0; e < R * VEC; e += 2) {
            const int r0 = e / VEC, v0 = e % VEC, r1 = (e + 1) / VEC, v1 = (e + 1) % VEC;
            float er0, er1;
            f2_get(f2_fma(f2(rg.zr[r0].get(v0), rg.zr[r1].get(v1)), nl, f2(b2r[v0], b2r[v1])), er0, er1);
            emax = fmaxf(emax, fmaxf(er0, er1));
            float t0, t1;
            f2_get(f2_add(f2(ex2_ftz(er0), ex2_ftz(er1)), one), t0, t1);
            const f32x2 rr = f2(rcp_ftz(t0), rcp_ftz(t1));
            const f32x2 x = f2_mul(rr, f2(l8[v0], l8[v1]));
            float x0, x1;
            f2_get(x, x0, x1);
            xmin = fminf(xmin, fminf(x0, x1));
            f32x2 a, nq;
            act_decay2(x, a, nq);
            f2_get(a, w.F[r0][v0], w.F[r1][v1]);
            if (side) {
                float ei0, ei1, q0, q1;
                f2_get(f2_fma(f2(rg.zi[r0].get(v0), rg.zi[r1].get(v1)), nl, f2(b2i[v0], b2i[v1])), ei0, ei1);
                emax = fmaxf(emax, fmaxf(ei0, ei1));
                f2_get(f2_add(f2(ex2_ftz(ei0), ex2_ftz(ei1)), one), t0, t1);
                const f32x2 ii = f2(rcp_ftz(t0), rcp_ftz(t1));
                f2_get(nq, q0, q1);
                qmin = fminf(qmin, fminf(-q0, -q1));
                const f32x2 nrf = f2(-rsqrt_ftz(-q0), -rsqrt_ftz(-q1));  // -1/f
                const f32x2 f = f2_mul(nq, nrf);
                const f32x2 u = f2_mul(ii, f2(rg.x[r0].get(v0), rg.x[r1].get(v1)));
                const f32x2 h = f2(rg.hp[r0].get(v0), rg.hp[r1].get(v1));
                // K = a (h - u a / f);  -K r, its product with lam (1 - r)
                const f32x2 K = f2_mul(a, f2_fma(f2_mul(u, a), nrf, h));
                const f32x2 nr = f2_mul(rr, none);
                const f32x2 KR = f2_mul(K, nr);
                const f32x2 CR = f2_mul(f2_mul(KR, f2(lam[v0], lam[v1])), f2_add(nr, one));
                const f32x2 CI = f2_mul(f2_mul(f, u), f2_fma(ii, none, one));
                f2_get(f2_mul(f, ii), w.CX[r0][v0], w.CX[r1][v1]);
                f2_get(CI, w.CI[r0][v0], w.CI[r1][v1]);
                f2_get(KR, w.KR[r0][v0], w.KR[r1][v1]);
                f2_get(CR, w.CR[r0][v0], w.CR[r1][v1]);
            }
        }
        const bool gen = emax > kGateMaxExp || xmin < kDecayMinX || !(qmin > 0.f);
        bool any = gen || !(tc.cok && tc.t0 < g.T) || (p.h0 != nullptr && tc.t0 - (R - 1) <= 0);
#pragma unroll
        for (int r = 0; r < R; ++r) any = any || rg.rs[r] != 0;
        if (any) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t t = tc.t0 - r;
                const bool ok = tc.cok && t < g.T, reset = rg.rs[r] != 0;
                const bool first = ok && t == 0 && p.h0 != nullptr;  // h0 is fp32
                if (ok && !reset && !gen && !first) continue;
                float hp[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) hp[v] = rg.hp[r].get(v);
                if (first) load_vec<float, VEC>(p.h0 + tc.c, hp);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float rr = act_sigmoid(rg.zr[r].get(v) + br[v]);
                    const float ii = act_sigmoid(rg.zi[r].get(v) + bi[v]);
                    float a, q;
                    act_decay(-lam[v] * rr, a, q);
                    // where the decay is 1 to the last bit (q = 0) its gradient is
                    // 0: K's pole is cancelled by r (1-r) -> 0
                    const float rf = q > 0.f ? rsqrt_ftz(q) : q;
                    const float f = reset ? 1.f : q * rf;
                    const float u = ii * rg.x[r].get(v);
                    const float K = reset || q == 0.f ? 0.f : a * (hp[v] - u * a * rf);
                    w.F[r][v] = ok ? (reset ? 0.f : a) : 1.f;
                    w.CX[r][v] = f * ii;
                    w.CI[r][v] = f * u * (1.f - ii);
                    w.KR[r][v] = -K * rr;
                    w.CR[r][v] = lam[v] * (w.KR[r][v] * (1.f - rr));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                // rows outside hold dh = 0 and F = 1
                B[v] = w.F[r][v] * (rg.dh[r].get(v) + B[v]);
                A[v] *= w.F[r][v];
            }
    }
    __device__ static void finish(const Params& p, const Geom& g, const TileCoord& tc,
                                  const Regs& rg, Work& w, float (&s)[VEC], Smem& xs, Acc& acc) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        float sum[3][VEC];
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) sum[k][v] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t t = tc.t0 - r;
            const bool ok = tc.cok && t < g.T;
            float dx[VEC], dzr[VEC], dzi[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float d = rg.dh[r].get(v) + s[v];
                dx[v] = d * w.CX[r][v];
                dzr[v] = d * w.CR[r][v];
                dzi[v] = d * w.CI[r][v];
                if (ok) {
                    sum[0][v] += d * w.KR[r][v];
                    sum[1][v] += dzr[v];
                    sum[2][v] += dzi[v];
                }
                s[v] = w.F[r][v] * d;
            }
            if (ok) {
                store_vec<S, VEC>(p.dx + t * g.C + tc.c, dx);
                store_vec<S, VEC>(p.dzr + t * g.C + tc.c, dzr);
                store_vec<S, VEC>(p.dzi + t * g.C + tc.c, dzi);
            }
        }
        if (tc.tchunk == 0 && warp == NW - 1 && p.dh0 != nullptr && tc.cok)
            store_vec<float, VEC>(p.dh0 + tc.c, s);
        const int64_t arr = g.n_chunks * g.C;
        float* out = p.partials + tc.tchunk * g.C + tc.c;
        if (tc.acc_run) {
            // a run of tiles of these channels through this CTA (see the SRU
            // backward pass): zeros but for the run's last tile
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc.s[k][v] += sum[k][v];
            if (!tc.acc_flush) {
                if (warp == 0 && tc.cok) {
#pragma unroll
                    for (int k = 0; k < 3; ++k)
#pragma unroll
                        for (int v = 0; v < VEC; ++v) out[k * arr + v] = 0.f;
                }
                return;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    sum[k][v] = acc.s[k][v];
                    acc.s[k][v] = 0.f;
                }
        }
        csync<NW>();  // every warp is past its reads of the previous tile's sums
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) xs.ps[k][warp][lane][v] = sum[k][v];
        csync<NW>();
        if (warp == 0 && tc.cok) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float t = 0.f;
#pragma unroll
                    for (int ww = 0; ww < NW; ++ww) t += xs.ps[k][ww][lane][v];
                    out[k * arr + v] = t;
                }
        }
    }
    __device__ static void at_exit(const Params&, Smem&, Acc&) {}
};

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

template <typename S, bool VP, int M>
using GlrFwdOpT = GlrFwdOp<S, kvec(sizeof(S) == 2, VP), kcfg(OP_GLR_FWD, sizeof(S) == 2, M).NW,
                           kcfg(OP_GLR_FWD, sizeof(S) == 2, M).R>;
template <typename S, bool VP, int M>
using GlrBwdOpT = GlrBwdOp<S, kvec(sizeof(S) == 2, VP), kcfg(OP_GLR_BWD, sizeof(S) == 2, M).NW,
                           kcfg(OP_GLR_BWD, sizeof(S) == 2, M).R>;

template <typename S, bool VP>
static cudaError_t glr_fwd_t(const GlrIn& in, const float* h0, void* h, float* h_last,
                             const Geom& g, const Carry& cr, cudaStream_t s) {
    return launch_persist<GlrFwdOpT<S, VP, CARRY_CHAIN>, GlrFwdOpT<S, VP, CARRY_WALK>,
                          GlrFwdOpT<S, VP, TILE_TMA>, kcfg(OP_GLR_FWD, sizeof(S) == 2, TILE_TMA).ST>(
        {(const S*)in.x, (const S*)in.zr, (const S*)in.zi, in.lam, in.br, in.bi, in.reset, h0, (S*)h,
         h_last, g.C / g.D},
        g, cr, s);
}

template <typename S, bool VP>
static cudaError_t glr_bwd_t(const GlrIn& in, const float* h0, const void* h, const void* dh,
                             const float* dh_last, void* dx, void* dzr, void* dzi, float* dh0,
                             float* partials, const Geom& g, const Carry& cr, cudaStream_t s) {
    return launch_persist<GlrBwdOpT<S, VP, CARRY_CHAIN>, GlrBwdOpT<S, VP, CARRY_WALK>,
                          GlrBwdOpT<S, VP, TILE_TMA>, kcfg(OP_GLR_BWD, sizeof(S) == 2, TILE_TMA).ST>(
        {(const S*)in.x, (const S*)in.zr, (const S*)in.zi, in.lam, in.br, in.bi, in.reset, h0,
         (const S*)h, (const S*)dh, dh_last, (S*)dx, (S*)dzr, (S*)dzi, dh0, partials, g.C / g.D},
        g, cr, s);
}

cudaError_t launch_glr_fwd(int dtype, bool vec, const GlrIn& in, const float* h0, void* h,
                           float* h_last, const Geom& g, const Carry& cr, cudaStream_t s) {
    if (dtype == 0)
        return vec ? glr_fwd_t<float, true>(in, h0, h, h_last, g, cr, s)
                   : glr_fwd_t<float, false>(in, h0, h, h_last, g, cr, s);
    return vec ? glr_fwd_t<__nv_bfloat16, true>(in, h0, h, h_last, g, cr, s)
               : glr_fwd_t<__nv_bfloat16, false>(in, h0, h, h_last, g, cr, s);
}

cudaError_t launch_glr_bwd(int dtype, bool vec, const GlrIn& in, const float* h0, const void* h,
                           const void* dh, const float* dh_last, void* dx, void* dzr, void* dzi,
                           float* dh0, float* partials, const Geom& g, const Carry& cr,
                           cudaStream_t s) {
    if (dtype == 0)
        return vec ? glr_bwd_t<float, true>(in, h0, h, dh, dh_last, dx, dzr, dzi, dh0, partials, g, cr, s)
                   : glr_bwd_t<float, false>(in, h0, h, dh, dh_last, dx, dzr, dzi, dh0, partials, g, cr, s);
    return vec ? glr_bwd_t<__nv_bfloat16, true>(in, h0, h, dh, dh_last, dx, dzr, dzi, dh0, partials, g,
                                                cr, s)
               : glr_bwd_t<__nv_bfloat16, false>(in, h0, h, dh, dh_last, dx, dzr, dzi, dh0, partials, g,
                                                 cr, s);
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
