// adamw_kernels.cu -- one AdamW step over many tensors in one launch, with the
// moments in fp32 or in 8 bits.
//
//   g' = gscale g,  m = b1 m + (1-b1) g',  v = b2 v + (1-b2) g'^2,
//   p = (1 - lr wd) p - (lr / (1-b1^t)) m / (sqrt(v / (1-b2^t)) + eps),
//   copy = p in bf16 (optional: the weights the next forward pass reads).
// Weights are fp32, gradients fp32 or bf16.
//
// 8 bits: blocks of 256 consecutive elements of a tensor share a scale, the
// largest magnitude of the block, and the codes q stand for rooted values, so
// that small magnitudes keep a relative accuracy:
//   m = scale sign(q) (q/127)^2,  q in -127 .. 127;   v = scale (q/255)^4.
// A moving average with b2 = 0.999 moves by less than a code step per call, so
// rounding to the nearest code would freeze it; the codes are rounded up or down
// with the probability that is right in the mean, by 16 bits of a hash of
// (element, tensor, seed): reproducible, and nothing is kept between calls.  A
// positive v never becomes 0 (the step divides by its root).  The codes are
// chosen with separately rounded IEEE operations (no contraction), so that they
// are the same wherever they are computed.  Where a block's scale is below 2^-120 (fp32
// holds no reciprocal below 2^-128), the block is taken times 2^64 first, which is
// exact: a moment that fades, or a first gradient of 1e-20, keeps its zeros at zero.
//
// Bytes bound it: each element of p, g, m, v crosses HBM once each way.  A
// launch takes up to kAdamTensors tensors, whose pointers travel in the kernel's
// arguments (no copy to the device, nothing to keep for a graph); a CTA finds
// its tensor by binary search over the chunk counts.  Measured: 128M elements in
// 160 tensors, bf16 gradients and copies, 546 us = 6.9 TB/s (copy 6.78); 8-bit
// moments, 64M elements in 90 tensors, fp32 gradients, 198 us = 5.4 TB/s, and their
// values written out 99 us = 6.8 TB/s.
#include "lr_act.cuh"
#include "lr_launch.h"

namespace lrs {

constexpr int kAdamChunk = 4096;  // elements of a CTA: 256 threads x 16

struct AdamTable {
    AdamTensor t[kAdamTensors];
    uint32_t first[kAdamTensors + 1];  // first chunk of each tensor
    int n;
    int base;  // the first tensor's index in the call (the hash)
};

__device__ __forceinline__ int adam_find(const AdamTable& tb, uint32_t chunk) {
    int lo = 0, hi = tb.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tb.first[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename G, int VEC>
__device__ __forceinline__ void adam_chunk(const AdamTensor& t, int64_t lo, int64_t hi,
                                           const AdamHyper& h, float gs) {
    const G* gp = (const G*)t.g;
    float* mp = (float*)t.m;
    float* vp = (float*)t.v;
    // hi - lo is a multiple of VEC on the vector path
    for (int64_t i = lo + (int64_t)threadIdx.x * VEC; i < hi; i += 256 * VEC) {
        Pack<G, VEC> pg;
        pg.load(gp + i);
        // updated in place: ordinary loads (load_shared is one), not the
        // read-only path
        Pack<float, VEC> pp, pm, pv;
        pp.load_shared(t.p + i);
        pm.load_shared(mp + i);
        pv.load_shared(vp + i);
        float p[VEC], m[VEC], v[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float g = pg.get(k) * gs;
            // beta1 and 1 - beta1 to twice the bits: where the terms cancel, m is
            // small against its root of v, and their rounding would show
            m[k] = fmaf(h.b1, pm.get(k), fmaf(h.c1, g, fmaf(h.b1_lo, pm.get(k), h.c1_lo * g)));
            v[k] = fmaf(h.b2, pv.get(k), fmaf(h.c2 * g, g, h.b2_lo * pv.get(k)));
            const float q = __fdiv_rn(m[k], fmaf(__fsqrt_rn(v[k]), h.rk2, h.eps));
            p[k] = fmaf(-h.step, q, fmaf(-h.step_lo, q, h.decay * pp.get(k)));
        }
        store_vec<float, VEC>(t.p + i, p);
        store_vec<float, VEC>(mp + i, m);
        store_vec<float, VEC>(vp + i, v);
        if (t.copy) store_vec<__nv_bfloat16, VEC>((__nv_bfloat16*)t.copy + i, p);
    }
}

template <typename G>
__global__ void __launch_bounds__(256)
    k_adamw(const __grid_constant__ AdamTable tb, const AdamHyper h, const float* __restrict__ gscale) {
    const uint32_t chunk = blockIdx.x;
    const int ti = adam_find(tb, chunk);
    const AdamTensor t = tb.t[ti];
    const float gs = gscale ? __ldg(gscale) : 1.f;
    const int64_t lo = (int64_t)(chunk - tb.first[ti]) * kAdamChunk;
    const int64_t hi = lo + kAdamChunk < t.n ? lo + kAdamChunk : t.n;
    if (t.vec) {
        const int64_t mid = lo + ((hi - lo) & ~(int64_t)3);
        adam_chunk<G, 4>(t, lo, mid, h, gs);
        adam_chunk<G, 1>(t, mid, hi, h, gs);
    } else {
        adam_chunk<G, 1>(t, lo, hi, h, gs);
    }
}

// ------------------------------------------------------------- 8-bit moments

// 32 mixed bits of (element, tensor, seed): two rounds of multiply and
// xor-shift; the constants are the fractional bits of the roots of 3, 2 and 5
// (and the golden ratio), made odd.
__device__ __forceinline__ uint32_t adam_hash(uint32_t i, uint32_t key) {
    uint32_t x = i + key;
    x = (x ^ (x >> 16)) * 0x6A09E667u;
    x = (x ^ (x >> 15)) * 0x3C6EF373u;
    return x ^ (x >> 16);
}
// Small integers as floats and back without the conversion instructions, which
// issue at a quarter of the rate of the others and were what bound this kernel: a
// byte b under the exponent of 2^23 is the float 2^23 + b; 16 bits under that of
// 1 are 1 + u / 2^16 (unit16); and adding 2^23 rounding towards zero leaves floor(x) in the
// low bits of the sum (0 <= x < 2^23).
__device__ __forceinline__ float byte_float(uint32_t w, int k, float bias) {
    return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u + (uint32_t)k)) - bias;
}
__device__ __forceinline__ float unit16(uint32_t u16) { return __uint_as_float(0x3F800000u | u16 << 7); }

// A sum of pairs, each of its terms rounded by itself: the compiler fuses
// mul.rn.f32x2 into an add.f32x2 that follows (seen in the results), so the
// additions after products are single ones.
__device__ __forceinline__ void add_apart(f32x2 a, f32x2 b, float& x, float& y) {
    float a0, a1, b0, b1;
    f2_get(a, a0, a1);
    f2_get(b, b0, b1);
    x = __fadd_rn(a0, b0);
    y = __fadd_rn(a1, b1);
}

__device__ __forceinline__ f32x2 adam_decode_m(float q0, float q1, f32x2 scale) {
    float t0, t1;
    f2_get(f2_mul(f2(q0, q1), f2(1.f / 127.f)), t0, t1);
    return f2_mul(f2(__fmul_rn(t0, fabsf(t0)), __fmul_rn(t1, fabsf(t1))), scale);
}
__device__ __forceinline__ f32x2 adam_decode_v(float q0, float q1, f32x2 scale) {
    f32x2 t = f2_mul(f2(q0, q1), f2(1.f / 255.f));
    t = f2_mul(t, t);
    return f2_mul(f2_mul(t, t), scale);
}

// A warp's next block on its way into shared memory: each lane copies what it will
// read itself, so that a wait on its own copies is all there is to wait for.
template <typename G>
struct A8Stage {
    float4 p[2][32];
    struct alignas(4 * sizeof(G)) Quad { Pack<G, 4> v; } g[2][32];
    uint32_t m[2][32], v[2][32];
};
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}
template <typename G>
__device__ __forceinline__ void adam8_fetch(const AdamTensor& t, int64_t blk, A8Stage<G>& st) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = blk * 256 + h * 128 + lane * 4;
        if (!t.vec || t.n - i < 4) continue;  // read in place
        copy_async<16>(&st.p[h][lane], t.p + i);
        copy_async<4 * sizeof(G)>(&st.g[h][lane], (const G*)t.g + i);
        copy_async<4>(&st.m[h][lane], (const uint8_t*)t.m + i);
        copy_async<4>(&st.v[h][lane], (const uint8_t*)t.v + i);
    }
}

// With F = 2^23 + floor(x - 1), x + (kHalfPast - F) is the fraction of x less 1/2,
// exactly.
constexpr float kHalfPast = 8388606.5f;
constexpr float kTinyScale = 0x1p-120f;

// The low byte of each of four floats, and 0xFF for each that is negative.
__device__ __forceinline__ uint32_t low_bytes(const float* f) {
    const uint32_t lo = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0040);
    return __byte_perm(lo, __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t sign_bytes(const float* f) {
    uint32_t lo, hi;  // selector nibbles B and F: the sign of byte 3 of either word, eight times
    asm("prmt.b32 %0, %1, %2, 0x00FB;" : "=r"(lo) : "r"(__float_as_uint(f[0])), "r"(__float_as_uint(f[1])));
    asm("prmt.b32 %0, %1, %2, 0x00FB;" : "=r"(hi) : "r"(__float_as_uint(f[2])), "r"(__float_as_uint(f[3])));
    return __byte_perm(lo, hi, 0x5410);
}

// One warp per block of 256 elements, four consecutive ones of each half a lane,
// worked on in pairs.  About 100 instructions an element (7 more with the codes put
// together one by one; IEEE roots throughout cost another 17), issue slots 84% busy.
// What it took for 64M elements, fp32 gradients: eight consecutive elements a lane,
// two accesses to every sector, 290 us; this layout 239 with three CTAs an SM, 224
// with four (64 registers; five spill: 269); chunks of 4096 209 (of 16384 216, of
// 32768 227); the codes packed by bytes 197, 5.5 TB/s.
template <typename G>
__device__ __forceinline__ void adam8_block(const AdamTensor& t, int64_t blk, const A8Stage<G>& st, float sm, float sv,
                                            const AdamHyper& h, float gs, uint32_t key) {
    const int lane = threadIdx.x & 31;
    const int64_t i0 = blk * 256 + lane * 4;
    uint8_t* mq = (uint8_t*)t.m;  // int8 codes
    uint8_t* vq = (uint8_t*)t.v;
    float p[8], g[8];
    uint32_t cm[2], cv[2];
    int n[2];  // elements inside the tensor
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = i0 + h * 128;
        n[h] = t.n - i >= 4 ? 4 : t.n > i ? (int)(t.n - i) : 0;
        if (t.vec && n[h] == 4) {
            const float4 a = st.p[h][lane];
            p[4 * h] = a.x; p[4 * h + 1] = a.y; p[4 * h + 2] = a.z; p[4 * h + 3] = a.w;
            const Pack<G, 4> gg = st.g[h][lane].v;
#pragma unroll
            for (int k = 0; k < 4; ++k) g[4 * h + k] = gg.get(k);
            cm[h] = st.m[h][lane];
            cv[h] = st.v[h][lane];
        } else {
            cm[h] = cv[h] = 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                p[4 * h + k] = g[4 * h + k] = 0.f;
                if (k >= n[h]) continue;
                p[4 * h + k] = t.p[i + k];
                Pack<G, 1> g1;
                g1.load((const G*)t.g + i + k);
                g[4 * h + k] = g1.get(0);
                cm[h] |= (uint32_t)mq[i + k] << (8 * k);
                cv[h] |= (uint32_t)vq[i + k] << (8 * k);
            }
        }
        cm[h] ^= 0x80808080u;  // signed codes, biased
    }
    // the new moments
    float m[8], v[8];
    float tm = 0.f, tv = 0.f;  // the block's new scales
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const uint32_t wm = cm[k >> 2], wv = cv[k >> 2];
        const f32x2 m0 = adam_decode_m(byte_float(wm, k & 3, 8388736.f), byte_float(wm, (k & 3) + 1, 8388736.f), f2(sm));
        const f32x2 v0 = adam_decode_v(byte_float(wv, k & 3, 8388608.f), byte_float(wv, (k & 3) + 1, 8388608.f), f2(sv));
        const f32x2 gg = f2_mul(f2(g[k], g[k + 1]), f2(gs));
        add_apart(f2_mul(m0, f2(h.b1)), f2_mul(gg, f2(h.c1)), m[k], m[k + 1]);
        add_apart(f2_mul(v0, f2(h.b2)), f2_mul(f2_mul(gg, gg), f2(h.c2)), v[k], v[k + 1]);
        tm = fmaxf(tm, fmaxf(fabsf(m[k]), fabsf(m[k + 1])));
        tv = fmaxf(tv, fmaxf(v[k], v[k + 1]));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, off));
        tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, off));
    }
    if (lane == 0) {
        t.ms[blk] = tm;
        t.vs[blk] = tv;
    }
    tv = fminf(tv, 0x1.fffffep127f);  // beside an infinite v the others keep their roots
    float step = h.step, rk2 = h.rk2;
    if (__builtin_expect(!(fminf(tm, tv) >= kTinyScale), 0)) {
        const bool um = tm < kTinyScale, uv = tv < kTinyScale;
        tm *= um ? 0x1p64f : 1.f;
        tv *= uv ? 0x1p64f : 1.f;
        step *= um ? 0x1p-64f : 1.f;  // it takes the block's m
        rk2 *= uv ? 0x1p-32f : 1.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            m[k] *= um ? 0x1p64f : 1.f;
            v[k] *= uv ? 0x1p64f : 1.f;
        }
    }
    const float im = tm > 0.f ? __fdiv_rn(1.f, tm) : 0.f, iv = tv > 0.f ? __fdiv_rn(1.f, tv) : 0.f;
    // sqrt(v) = sqrt(v / scale) sqrt(scale): the first root is the code's too
    const float rv = sqrtf(tv) * rk2;
    uint32_t qm[2], qv[2];
#pragma unroll
    for (int h4 = 0; h4 < 2; ++h4) {
        float fa[4], fb[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const int k = 4 * h4 + j;
            float rm[2], r2[2], root[2], a[2], b[2], um[2], uv[2], da[2], db[2];
            f2_get(f2_mul(f2(v[k], v[k + 1]), f2(iv)), r2[0], r2[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t u = adam_hash((uint32_t)(i0 + h4 * 128 + j + e), key);
                um[e] = unit16(u >> 16);
                uv[e] = unit16(u & 0xffffu);
                rm[e] = __fmul_rn(fabsf(m[k + e]), im);
                root[e] = sqrt_ftz(r2[e]);
                a[e] = fmaf(sqrt_ftz(rm[e]), 127.f, um[e]);  // one more than the code's sum
                b[e] = fmaf(sqrt_ftz(root[e]), 255.f, uv[e]);
                fa[j + e] = __fadd_rz(a[e], 8388607.f);
                fb[j + e] = __fadd_rz(b[e], 8388607.f);
            }
            f2_get(f2_add(f2(a[0], a[1]), f2_add(f2(kHalfPast), f2(-fa[j], -fa[j + 1]))), da[0], da[1]);
            f2_get(f2_add(f2(b[0], b[1]), f2_add(f2(kHalfPast), f2(-fb[j], -fb[j + 1]))), db[0], db[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // The roots are good to a few 2^-23: a and b to 6e-5 and 1.4e-4.  Where
                // that does not settle the code (or v / scale is subnormal: flushed; or
                // NaN), in about one element of 1500, the IEEE roots do.
                if (!(fabsf(da[e]) < 0.5f - 1e-4f && fabsf(db[e]) < 0.5f - 2e-4f && r2[e] >= 1.17549435e-38f)) {
                    root[e] = __fsqrt_rn(r2[e]);
                    const float x = __fadd_rn(__fmul_rn(__fsqrt_rn(rm[e]), 127.f), um[e] - 1.f);
                    const float y = __fadd_rn(__fmul_rn(__fsqrt_rn(root[e]), 255.f), uv[e] - 1.f);
                    fa[j + e] = fminf(__fadd_rz(x, 8388608.f), 8388608.f + 127.f);
                    fb[j + e] = fminf(__fadd_rz(y, 8388608.f), 8388608.f + 255.f);
                    // a ratio that fp32 holds in part or not at all: its root is in range
                    if (r2[e] < 1.17549435e-38f && v[k + e] > 0.f) root[e] = __fdiv_rn(__fsqrt_rn(v[k + e]), sqrtf(tv));
                }
                if (v[k + e] > 0.f) fb[j + e] = fmaxf(fb[j + e], 8388609.f);
                p[k + e] = fmaf(-step, __fdividef(m[k + e], fmaf(root[e], rv, h.eps)), h.decay * p[k + e]);
            }
        }
        // the four codes of each: the floats' low bytes, m's with its sign (bytes that
        // are biased by 128 stay positive, so the sums below carry nothing over)
        const uint32_t mag = low_bytes(fa), neg = sign_bytes(m + 4 * h4);
        qm[h4] = (0x80808080u + (mag & ~neg) - (mag & neg)) ^ 0x80808080u;
        qv[h4] = low_bytes(fb);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = i0 + h * 128;
        const float* ph = p + 4 * h;
        if (t.vec && n[h] == 4) {
            *reinterpret_cast<float4*>(t.p + i) = make_float4(ph[0], ph[1], ph[2], ph[3]);
            *reinterpret_cast<uint32_t*>(mq + i) = qm[h];
            *reinterpret_cast<uint32_t*>(vq + i) = qv[h];
            if (t.copy)
                *reinterpret_cast<uint2*>((__nv_bfloat16*)t.copy + i) = make_uint2(bf_pack(ph[0], ph[1]), bf_pack(ph[2], ph[3]));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= n[h]) continue;
                t.p[i + k] = ph[k];
                mq[i + k] = (uint8_t)(qm[h] >> (8 * k));
                vq[i + k] = (uint8_t)(qv[h] >> (8 * k));
                if (t.copy) ((__nv_bfloat16*)t.copy)[i + k] = __float2bfloat16_rn(ph[k]);
            }
        }
    }
}

template <typename G>
__global__ void __launch_bounds__(256, 4)
    k_adamw8(const __grid_constant__ AdamTable tb, const AdamHyper h, const float* __restrict__ gscale,
             uint32_t seed) {
    __shared__ A8Stage<G> st[8][2];
    const uint32_t chunk = blockIdx.x;
    const int ti = adam_find(tb, chunk), warp = threadIdx.x >> 5;
    const AdamTensor t = tb.t[ti];
    const float gs = gscale ? __ldg(gscale) : 1.f;
    const uint32_t key = (uint32_t)(tb.base + ti) * 0x9E3779B1u + seed * 0xBB67AE85u;
    const int64_t lo = (int64_t)(chunk - tb.first[ti]) * (kAdamChunk / 256);
    const int64_t nb = (t.n + 255) / 256, end = nb < lo + kAdamChunk / 256 ? nb : lo + kAdamChunk / 256;
    int64_t blk = lo + warp;
    if (blk >= end) return;
    adam8_fetch<G>(t, blk, st[warp][0]);
    asm volatile("cp.async.commit_group;" ::: "memory");
    float sm = t.ms[blk], sv = t.vs[blk];
    for (int cur = 0; blk < end; blk += 8, cur ^= 1) {
        float sm1 = 0.f, sv1 = 0.f;
        if (blk + 8 < end) {  // the next block's copies fly while this one is worked on
            adam8_fetch<G>(t, blk + 8, st[warp][cur ^ 1]);
            sm1 = t.ms[blk + 8];
            sv1 = t.vs[blk + 8];
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        adam8_block<G>(t, blk, st[warp][cur], sm, sv, h, gs, key);
        sm = sm1;
        sv = sv1;
    }
}

// The values that 8-bit moments stand for (fp32), to be saved or looked at:
// t.p = where m goes, t.copy = where v goes (fp32), t.m / t.v / t.ms / t.vs the
// codes and scales.
__global__ void __launch_bounds__(256) k_adamw8_values(const __grid_constant__ AdamTable tb) {
    const uint32_t chunk = blockIdx.x;
    const int ti = adam_find(tb, chunk);
    const AdamTensor t = tb.t[ti];
    const int64_t lo = (int64_t)(chunk - tb.first[ti]) * kAdamChunk;
    const int64_t hi = lo + kAdamChunk < t.n ? lo + kAdamChunk : t.n;
    const int8_t* mq = (const int8_t*)t.m;
    const uint8_t* vq = (const uint8_t*)t.v;
    float* vo = (float*)t.copy;
    auto one = [&](int64_t i) {
        float x;
        f2_get(adam_decode_m((float)mq[i], 0.f, f2(__ldg(t.ms + (i >> 8)))), t.p[i], x);
        f2_get(adam_decode_v((float)vq[i], 0.f, f2(__ldg(t.vs + (i >> 8)))), vo[i], x);
    };
    if (t.vec) {
        const int64_t mid = lo + ((hi - lo) & ~(int64_t)3);
        for (int64_t i = lo + (int64_t)threadIdx.x * 4; i < mid; i += 1024) {
            const uint32_t cm = *reinterpret_cast<const uint32_t*>(mq + i);
            const uint32_t cv = *reinterpret_cast<const uint32_t*>(vq + i);
            const float sm = __ldg(t.ms + (i >> 8)), sv = __ldg(t.vs + (i >> 8));
            const uint32_t wm = cm ^ 0x80808080u;
            float m[4], v[4];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                f2_get(adam_decode_m(byte_float(wm, k, 8388736.f), byte_float(wm, k + 1, 8388736.f), f2(sm)), m[k], m[k + 1]);
                f2_get(adam_decode_v(byte_float(cv, k, 8388608.f), byte_float(cv, k + 1, 8388608.f), f2(sv)), v[k], v[k + 1]);
            }
            store_vec<float, 4>(t.p + i, m);
            store_vec<float, 4>(vo + i, v);
        }
        for (int64_t i = mid + threadIdx.x; i < hi; i += 256) one(i);
    } else {
        for (int64_t i = lo + threadIdx.x; i < hi; i += 256) one(i);
    }
}

cudaError_t launch_adamw(AdamKind kind, int gdtype, const AdamTensor* t, int64_t n_tensors,
                         const AdamHyper& h, const float* gscale, uint32_t seed, cudaStream_t s) {
    int64_t i = 0;
    while (i < n_tensors) {
        AdamTable tb;
        tb.n = 0;
        tb.base = (int)i;
        uint64_t chunks = 0;
        for (; i < n_tensors && tb.n < kAdamTensors; ++i) {
            const uint64_t c = (uint64_t)((t[i].n + kAdamChunk - 1) / kAdamChunk);
            if (chunks + c > 0x7fffffffull) {
                if (tb.n == 0) return cudaErrorInvalidValue;
                break;
            }
            // an empty tensor takes an entry without a chunk: the hash's
            // tensor index is the index in the call
            tb.t[tb.n] = t[i];
            tb.first[tb.n] = (uint32_t)chunks;
            chunks += c;
            ++tb.n;
        }
        tb.first[tb.n] = (uint32_t)chunks;
        if (chunks == 0) continue;
        const unsigned grid = (unsigned)chunks;
        if (kind == ADAM_VALUES) k_adamw8_values<<<grid, 256, 0, s>>>(tb);
        else if (kind == ADAM_8BIT && gdtype == 0) k_adamw8<float><<<grid, 256, 0, s>>>(tb, h, gscale, seed);
        else if (kind == ADAM_8BIT) k_adamw8<__nv_bfloat16><<<grid, 256, 0, s>>>(tb, h, gscale, seed);
        else if (gdtype == 0) k_adamw<float><<<grid, 256, 0, s>>>(tb, h, gscale);
        else k_adamw<__nv_bfloat16><<<grid, 256, 0, s>>>(tb, h, gscale);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace lrs
