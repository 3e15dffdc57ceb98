// lr_act.cuh -- the activations of the fused producers and epilogues: the
// logistic sigmoid (SRU gates, page [P1] "CUDA并行化RNN训练：从O(T)到O(log T)的
// 工程实践与参数调优", SRU paragraph; LSTM gates), tanh (SRU output and cell
// gradient; LSTM candidate and output; DEER's diagonal tanh RNN, page [P4],
// section "核心原理") and e^x - 1 (DEER's ODE form, page [P4], section
// "监控与调优").
//
// Both are written from their exponential forms,
//     sigmoid(z) = 1 / (1 + 2^{-z log2 e}),
//     tanh(x)    = 1 - 2 r,  r = 1 / (2^{2 x log2 e} + 1),
// and the derivative of tanh from the same r, 1 - tanh^2 = 4 r (1 - r), free of
// the cancellation of 1 - tanh^2 where tanh saturates;
// with the power of two and the reciprocal taken from the hardware's
// approximate instructions (ex2.approx, rcp.approx) in their flush-to-zero
// forms: one instruction each, with no extra steps for subnormal results,
// which none of these forms needs (a subnormal power of two or reciprocal only
// occurs where the result has saturated to 0 or 1 anyway).  That is a few
// instructions per activation, which matters here: these kernels stream 24-40
// bytes per element, and with two to five activations per element the DEER,
// SRU and LSTM kernels are bound by instruction issue.  Both forms saturate
// correctly (an infinite power gives a reciprocal of 0), keep NaN, and have an
// absolute error of a few 1e-7 on the whole line (no cancellation issue for
// the absolute error near 0), well inside the 1e-5 tolerance the results are
// checked against; lr_test_activations exposes them to the test that bounds
// their error against fp64.
#pragma once

#include <cuda_runtime.h>

namespace lrs {

// 2^x and 1/x, hardware approximations (relative error about 2^-22), with
// subnormal results flushed to zero.
__device__ __forceinline__ float ex2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;       // log2(e)
constexpr float kTwoLog2e = 2.8853900817779268f;    // 2 log2(e)

__device__ __forceinline__ float act_sigmoid(float z) {
    return rcp_ftz(1.f + ex2_ftz(-kLog2e * z));
}

// tanh(x) keeps its sign for x < 0 (r > 1/2 there) and saturates to -1 (the
// power flushes to 0) and +1 (an infinite power gives r = 0).
__device__ __forceinline__ float act_tanh(float x) {
    return fmaf(-2.f, rcp_ftz(ex2_ftz(kTwoLog2e * x) + 1.f), 1.f);
}
// tanh(x), and in d its derivative 1 - tanh(x)^2.
__device__ __forceinline__ float act_tanh_d(float x, float& d) {
    const float r = rcp_ftz(ex2_ftz(kTwoLog2e * x) + 1.f);
    d = 4.f * fmaf(-r, r, r);
    return fmaf(-2.f, r, 1.f);
}
// tanh(x), and in q a quarter of its derivative, r (1 - r) with
// r = 1 / (e^{2x} + 1): a caller that scales the factor it multiplies the
// derivative by with 4 once (exact in fp32) saves a multiply per element and
// gets the same bits as 4 q times that factor.
__device__ __forceinline__ float act_tanh_q(float x, float& q) {
    const float r = rcp_ftz(ex2_ftz(kTwoLog2e * x) + 1.f);
    q = fmaf(-r, r, r);
    return fmaf(-2.f, r, 1.f);
}

// e^x - 1 without the cancellation of e^x - 1 near 0 (DEER's ODE form,
// exp(-G dt) and (1 - exp(-G dt)) / G): below |x| = 1/4 the Taylor series
// x (1 + x/2 (1 + x/3 (... (1 + x/8)))) -- its first omitted term, x^9/9!, is
// under 1e-11 |x| there -- and elsewhere e^x - 1 from the hardware
// exponential, where |e^x - 1| > 0.22 keeps the subtraction exact to a few
// ulp.  NaN stays NaN, -inf gives -1, +inf gives +inf.
__device__ __forceinline__ float act_expm1(float x) {
    if (fabsf(x) < 0.25f) {
        float p = fmaf(x, 0.125f, 1.f);
        p = fmaf(x * (1.f / 7.f), p, 1.f);
        p = fmaf(x * (1.f / 6.f), p, 1.f);
        p = fmaf(x * 0.2f, p, 1.f);
        p = fmaf(x * 0.25f, p, 1.f);
        p = fmaf(x * (1.f / 3.f), p, 1.f);
        p = fmaf(x * 0.5f, p, 1.f);
        return x * p;
    }
    return ex2_ftz(kLog2e * x) - 1.f;
}

// Square root and reciprocal square root, hardware approximations (relative
// error about 2^-23 and 2^-22), subnormals flushed to zero.
__device__ __forceinline__ float sqrt_ftz(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsqrt_ftz(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The decay of the gated linear recurrence, a = e^l for l <= 0, and
// q = 1 - a^2 without the cancellation where a is near 1 (long memories): with
// m = e^l - 1 by its Taylor series near 0, a = 1 + m and q = -m (2 + m).
// The series stops at l^7/7!: the first omitted term is under 4e-9 |l| at
// |l| = 1/4.  Below, the hardware exponential: q > 0.39 there.
__device__ __forceinline__ void act_decay(float l, float& a, float& q) {
    if (l > -0.25f) {
        float p = fmaf(l, 1.f / 7.f, 1.f);
        p = fmaf(l * (1.f / 6.f), p, 1.f);
        p = fmaf(l * 0.2f, p, 1.f);
        p = fmaf(l * 0.25f, p, 1.f);
        p = fmaf(l * (1.f / 3.f), p, 1.f);
        p = fmaf(l * 0.5f, p, 1.f);
        const float m = l * p;
        a = 1.f + m;
        q = -m * (2.f + m);
    } else {
        a = ex2_ftz(kLog2e * l);
        q = fmaf(-a, a, 1.f);
    }
}

// ---- two fp32 values in one 64-bit register (sm_100+: one instruction issues
// both operations, which is what a kernel bound by instruction issue counts).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 f2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f32x2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void f2_get(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 f2_fma(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 f2_mul(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 f2_add(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// act_decay for a pair, without a branch or the exponential, for l in [-4, 0]:
// x = l / 16, m = e^x - 1 by its series (the first omitted term is under
// 5e-8 |x|), then four times e^2x - 1 = (e^x - 1)(2 + (e^x - 1)).  The series runs
// on single values: its coefficients are immediate operands there, and as pairs
// would take a register pair each.  q = 1 - a^2 + 1e-30: positive for every
// decay, so that its root has no pole (1e-30 is below any q that a decay other
// than 1 has, and its root, 1e-15, below any state's last bit).
constexpr float kDecayMaxRate = 4.f;
__device__ __forceinline__ float expm1_16th(float x) {
    float p = fmaf(x, 1.f / 720.f, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    return fmaf(p * x, x, x);
}
__device__ __forceinline__ void act_decay2(f32x2 x, f32x2& a, f32x2& q) {
    const f32x2 one = f2(1.f), two = f2(2.f), none = f2(-1.f), ntwo = f2(-2.f), tiny = f2(1e-30f);
    float x0, x1;
    f2_get(x, x0, x1);
    f32x2 m = f2(expm1_16th(x0), expm1_16th(x1));
    m = f2_mul(m, f2_add(m, two));
    m = f2_mul(m, f2_add(m, two));
    m = f2_mul(m, f2_add(m, two));
    m = f2_mul(m, f2_add(m, two));
    a = f2_add(m, one);
    q = f2_fma(m, f2_fma(m, none, ntwo), tiny);
}

}  // namespace lrs
