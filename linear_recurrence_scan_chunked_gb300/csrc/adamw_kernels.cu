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
// are the same wherever they are computed.
//
// Bytes bound it: each element of p, g, m, v crosses HBM once each way.  A
// launch takes up to kAdamTensors tensors, whose pointers travel in the kernel's
// arguments (no copy to the device, nothing to keep for a graph); a CTA finds
// its tensor by binary search over the chunk counts.
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
__device__ __forceinline__ float adam_decode_m(int q, float scale) {
    const float t = __fmul_rn((float)q, 1.f / 127.f);
    return __fmul_rn(__fmul_rn(t, fabsf(t)), scale);
}
__device__ __forceinline__ float adam_decode_v(int q, float scale) {
    float t = __fmul_rn((float)q, 1.f / 255.f);
    t = __fmul_rn(t, t);
    return __fmul_rn(__fmul_rn(t, t), scale);
}

// One warp per block of 256 elements, 8 consecutive ones a lane.
template <typename G, bool VP>
__device__ __forceinline__ void adam8_block(const AdamTensor& t, int64_t blk, const AdamHyper& h,
                                            float gs, uint32_t key) {
    const int lane = threadIdx.x & 31;
    const int64_t i0 = blk * 256 + lane * 8;
    const int n = t.n - i0 >= 8 ? 8 : t.n > i0 ? (int)(t.n - i0) : 0;
    const G* gp = (const G*)t.g;
    int8_t* mq = (int8_t*)t.m;
    uint8_t* vq = (uint8_t*)t.v;
    const float sm = t.ms[blk], sv = t.vs[blk];
    float p[8], m[8], v[8];
    if (VP && n == 8) {
        const float4 a = *reinterpret_cast<const float4*>(t.p + i0);
        const float4 b = *reinterpret_cast<const float4*>(t.p + i0 + 4);
        p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
        p[4] = b.x; p[5] = b.y; p[6] = b.z; p[7] = b.w;
        const uint2 cm = *reinterpret_cast<const uint2*>(mq + i0);
        const uint2 cv = *reinterpret_cast<const uint2*>(vq + i0);
        Pack<G, 4> g0, g1;
        g0.load(gp + i0);
        g1.load(gp + i0 + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t wm = k < 4 ? cm.x : cm.y, wv = k < 4 ? cv.x : cv.y;
            m[k] = adam_decode_m((int)(int8_t)(wm >> (8 * (k & 3))), sm);
            v[k] = adam_decode_v((int)((wv >> (8 * (k & 3))) & 255u), sv);
            const float g = __fmul_rn(k < 4 ? g0.get(k & 3) : g1.get(k & 3), gs);
            m[k] = __fadd_rn(__fmul_rn(h.b1, m[k]), __fmul_rn(h.c1, g));
            v[k] = __fadd_rn(__fmul_rn(h.b2, v[k]), __fmul_rn(h.c2, __fmul_rn(g, g)));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            p[k] = m[k] = v[k] = 0.f;
            if (k >= n) continue;
            p[k] = t.p[i0 + k];
            Pack<G, 1> g1;
            g1.load(gp + i0 + k);
            const float g = __fmul_rn(g1.get(0), gs);
            m[k] = __fadd_rn(__fmul_rn(h.b1, adam_decode_m((int)mq[i0 + k], sm)), __fmul_rn(h.c1, g));
            v[k] = __fadd_rn(__fmul_rn(h.b2, adam_decode_v((int)vq[i0 + k], sv)),
                             __fmul_rn(h.c2, __fmul_rn(g, g)));
        }
    }
    float tm = 0.f, tv = 0.f;  // the block's new scales
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        tm = fmaxf(tm, fabsf(m[k]));
        tv = fmaxf(tv, v[k]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, off));
        tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, off));
    }
    const float im = tm > 0.f ? __fdiv_rn(1.f, tm) : 0.f, iv = tv > 0.f ? __fdiv_rn(1.f, tv) : 0.f;
    uint32_t qm[8], qv[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        p[k] = fmaf(-h.step, __fdividef(m[k], fmaf(sqrtf(v[k]), h.rk2, h.eps)), h.decay * p[k]);
        const uint32_t u = adam_hash((uint32_t)(i0 + k), key);
        const float um = (float)(u >> 16) * (1.f / 65536.f), uv = (float)(u & 0xffffu) * (1.f / 65536.f);
        float a = __fsqrt_rn(__fmul_rn(fabsf(m[k]), im));
        a = fminf(floorf(__fadd_rn(__fmul_rn(a, 127.f), um)), 127.f);
        float b = __fsqrt_rn(__fsqrt_rn(__fmul_rn(v[k], iv)));
        b = fminf(floorf(__fadd_rn(__fmul_rn(b, 255.f), uv)), 255.f);
        if (v[k] > 0.f && b < 1.f) b = 1.f;
        const int q = (int)a;
        qm[k] = (uint32_t)(m[k] < 0.f ? -q : q) & 255u;
        qv[k] = (uint32_t)(int)b & 255u;
    }
    if (VP && n == 8) {
        *reinterpret_cast<float4*>(t.p + i0) = make_float4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<float4*>(t.p + i0 + 4) = make_float4(p[4], p[5], p[6], p[7]);
        *reinterpret_cast<uint2*>(mq + i0) =
            make_uint2(qm[0] | qm[1] << 8 | qm[2] << 16 | qm[3] << 24, qm[4] | qm[5] << 8 | qm[6] << 16 | qm[7] << 24);
        *reinterpret_cast<uint2*>(vq + i0) =
            make_uint2(qv[0] | qv[1] << 8 | qv[2] << 16 | qv[3] << 24, qv[4] | qv[5] << 8 | qv[6] << 16 | qv[7] << 24);
        if (t.copy)
            *reinterpret_cast<uint4*>((__nv_bfloat16*)t.copy + i0) =
                make_uint4(bf_pack(p[0], p[1]), bf_pack(p[2], p[3]), bf_pack(p[4], p[5]), bf_pack(p[6], p[7]));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= n) continue;
            t.p[i0 + k] = p[k];
            mq[i0 + k] = (int8_t)qm[k];
            vq[i0 + k] = (uint8_t)qv[k];
            if (t.copy) ((__nv_bfloat16*)t.copy)[i0 + k] = __float2bfloat16_rn(p[k]);
        }
    }
    if (lane == 0) {
        t.ms[blk] = tm;
        t.vs[blk] = tv;
    }
}

template <typename G>
__global__ void __launch_bounds__(256)
    k_adamw8(const __grid_constant__ AdamTable tb, const AdamHyper h, const float* __restrict__ gscale,
             uint32_t seed) {
    const uint32_t chunk = blockIdx.x;
    const int ti = adam_find(tb, chunk);
    const AdamTensor t = tb.t[ti];
    const float gs = gscale ? __ldg(gscale) : 1.f;
    const uint32_t key = (uint32_t)(tb.base + ti) * 0x9E3779B1u + seed * 0xBB67AE85u;
    const int64_t lo = (int64_t)(chunk - tb.first[ti]) * (kAdamChunk / 256);
    const int64_t nb = (t.n + 255) / 256;
    for (int64_t blk = lo + (threadIdx.x >> 5); blk < nb && blk < lo + kAdamChunk / 256; blk += 8) {
        if (t.vec) adam8_block<G, true>(t, blk, h, gs, key);
        else adam8_block<G, false>(t, blk, h, gs, key);
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
    if (t.vec) {
        const int64_t mid = lo + ((hi - lo) & ~(int64_t)3);
        for (int64_t i = lo + (int64_t)threadIdx.x * 4; i < mid; i += 1024) {
            const uint32_t cm = *reinterpret_cast<const uint32_t*>(mq + i);
            const uint32_t cv = *reinterpret_cast<const uint32_t*>(vq + i);
            const float sm = __ldg(t.ms + (i >> 8)), sv = __ldg(t.vs + (i >> 8));
            float m[4], v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = adam_decode_m((int)(int8_t)(cm >> (8 * k)), sm);
                v[k] = adam_decode_v((int)((cv >> (8 * k)) & 255u), sv);
            }
            store_vec<float, 4>(t.p + i, m);
            store_vec<float, 4>(vo + i, v);
        }
        for (int64_t i = mid + threadIdx.x; i < hi; i += 256) {
            t.p[i] = adam_decode_m((int)mq[i], __ldg(t.ms + (i >> 8)));
            vo[i] = adam_decode_v((int)vq[i], __ldg(t.vs + (i >> 8)));
        }
    } else {
        for (int64_t i = lo + threadIdx.x; i < hi; i += 256) {
            t.p[i] = adam_decode_m((int)mq[i], __ldg(t.ms + (i >> 8)));
            vo[i] = adam_decode_v((int)vq[i], __ldg(t.vs + (i >> 8)));
        }
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
