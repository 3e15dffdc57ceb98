// lce_mma.cuh -- the matrix products of the cross entropy on the tensor cores
// (tcgen05.mma, bf16 operands, fp32 accumulators in TMEM).
//
// One kernel, three products: logits x W^T, g W and g^T x.  A pair of CTAs
// (cta_group::2, a cluster of two on neighbouring SMs) owns a 256 x TN tile of
// the result: each holds 128 rows of A, half of B and the accumulators of its
// 128 rows, so an operand byte in shared memory feeds twice the arithmetic of a
// single CTA's tile.  TN is 256; 128 or (K-major B) 64 where wider tiles would leave pairs idle.
// Per CTA: a producer thread keeps a ring of k-blocks of 64 in flight by TMA
// (128-byte swizzle), one thread of the pair's first CTA
// issues the MMAs, and eight warps read finished accumulators back and run the
// epilogue while the next tile accumulates in the other half of TMEM.
//
// The tensor cores add into their fp32 accumulators by truncation: a step of 16 shrinks
// a sum by about 5e-9 of itself where its terms have random signs (measured on the loss:
// 1.3e-6 over k = 4096) and by 6e-8 to 9e-8 where they have one sign (a confident row's
// logit: 1.5e-5 over k = 4096; a gradient over 131072 words: 7e-4).  So the loop is cut
// into chunks of k-blocks (kChunk for the logits of bf16 data, more for its gradients,
// fewer for fp32) whose accumulators the epilogue warps add up in registers, rounding
// to nearest.
//
// Operands are [rows][cols] matrices of bf16 planes: one plane for bf16 data,
// three for fp32 data split as a = a1 + a2 + a3 (8 bits of mantissa each), whose
// six leading products a_i b_j, i + j <= 4, give the fp32 product to 2^-24.  An
// operand is K-major when k runs along its rows' contiguous axis, MN-major when
// it runs across them; both come out of TMA in the layouts that the matrix
// descriptors name, so no product needs a transposed copy.
//
// Every wait is bounded: one that runs out records LR_ERR_TIMEOUT, the epilogue makes
// NaN of the results that it waited for, the other roles leave their loops, the pair
// meets, lets its copies land and frees its TMEM.
#pragma once

#include "lr_tma.cuh"

namespace lrs {
namespace mm {

constexpr int kTile = 256;       // rows of a pair's tile
constexpr int kHalf = 128;       // rows of A that a CTA holds
constexpr int kBlockK = 64;      // k-block: 128 bytes of bf16, the swizzle's width
constexpr int kOperandA = kHalf * kBlockK * 2;  // 16 KB: A of a stage
constexpr int kThreads = 320;    // producer warp, MMA warp, 8 epilogue warps
constexpr uint32_t kChunk = 16;  // k-blocks of a chunk: k = 1024, 3e-7 of a logit of random signs (fp32 planes: 2)
constexpr int kScratch = 32 * 33 * 4;  // bytes an epilogue warp may use

template <int TN>
struct Cfg {
    static constexpr int kHalfN = TN / 2;                      // rows of B that a CTA holds; columns of an epilogue warp
    static constexpr int kOperandB = kHalfN * kBlockK * 2;
    static constexpr int kStageBytes = kOperandA + kOperandB;  // of one CTA
    static constexpr int kStages = TN == 256 ? 6 : 8;          // 192 KB (TN = 64: 160 KB)
    static constexpr int kRing = kStages * kStageBytes;
    static constexpr int smem(bool scratch) { return kRing + 1024 + (scratch ? 8 * kScratch : 0); }
};

// What the products share: the tile grid and the k loop.
struct Shape {
    uint32_t tm, tn;        // tiles along the result's rows and columns
    uint32_t splits;        // parts of the k loop, each a tile of its own
    uint32_t kb;            // k-blocks of the whole loop
    uint32_t kb_split;      // k-blocks of a part
    uint32_t n_fast;        // neighbouring tiles along the columns (else along the rows)
    uint32_t a_mn, b_mn;    // MN-major operands
    uint64_t wait_ns;       // limit of a wait
    uint32_t stalled;       // test: no operand is loaded, so that every wait runs out
};

// Both CTAs of the pair, all threads.
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) { return cluster_map(p, rank); }

// 3-D box {x, y, plane} into this CTA's shared memory; the bytes count on the
// barrier at cluster address `bar` (the pair's first CTA's).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* m, int32_t x, int32_t y, int32_t z,
                                              uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint64_t* b, uint32_t parity, const uint32_t* err, uint64_t limit_ns) {
    if (mbar_try_wait_cluster(b, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait_cluster(b, parity)) return true;
        if ((n & 255u) == 0) {
            if (globaltimer_ns() - t0 > limit_ns) return false;
            if (ld_relaxed_u32(err) & ERRBIT_TIMEOUT) return false;
        }
    }
}

// ---- tcgen05
//
// TMEM is managed by a warp of each CTA of the pair together, and an instruction of one
// reaches the other's TMEM: the peer has to be running when either is issued, both have to
// hold their columns before one gives up its permit, and neither may end before both
// have given their columns back.  The pair meets at each of these points.  (With only the
// meeting before the columns are given back, one CTA in some 10^6 waited for its columns
// for ever while its peer had its own.  Taking them has no limit of its own.)
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                 : "memory");
}
__device__ __forceinline__ void tmem_permit_back() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The barrier at this offset in both CTAs completes when the MMAs issued so far have.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// 32 columns of this warp's 32 accumulator rows.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major: rows of 128 bytes,
// groups of 8 rows 1024 bytes apart.  MN-major: blocks of 64 elements (128 bytes)
// by 64 k-rows, groups of 8 k-rows 1024 bytes apart, blocks 8192 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn) {
    const uint64_t lead = mn ? 8192 >> 4 : 1;
    return (uint64_t)((addr >> 4) & 0x3fff) | lead << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// bf16 x bf16 -> fp32, 256 x tn.
__device__ __forceinline__ uint32_t instr_desc(bool a_mn, bool b_mn, int tn) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (uint32_t)(tn >> 3) << 17 |
           (uint32_t)(kTile >> 4) << 24;
}

// The plane pairs of fp32 data, smallest products first.  A k-block's planes take
// a stage each and are loaded once for the six products.
__device__ constexpr int pair_a(int p) { return (0x001012 >> (4 * p)) & 3; }
__device__ constexpr int pair_b(int p) { return (0x010210 >> (4 * p)) & 3; }

struct Tile {
    uint32_t m, n, split;
};
__device__ __forceinline__ Tile tile_of(const Shape& s, uint32_t t) {
    Tile r;
    const uint32_t per = s.tm * s.tn;
    r.split = t / per;
    t -= r.split * per;
    if (s.n_fast) {
        r.m = t / s.tn;
        r.n = t - r.m * s.tn;
    } else {
        r.n = t / s.tm;
        r.m = t - r.n * s.tm;
    }
    return r;
}

// k-blocks of a tile, and of a chunk.  Three planes issue six products a k-block.
// Relative errors and time, fp32 loss and gradients: 563 x 2524, V 15623, chunks of
// 3: loss 3.2e-7, dx 6.4e-7, 950 us; of 2: 1.8e-7, 4.1e-7, 967 us; of 1: 5e-8, 1.9e-7,
// 1045 us (plain fp32 products: 1e-7 to 6e-7).
__host__ __device__ constexpr uint32_t chunk_of(int planes) { return planes == 1 ? kChunk : 2; }
__device__ __forceinline__ uint32_t tile_steps(const Shape& s, const Tile& t) {
    const uint32_t k0 = t.split * s.kb_split;
    const uint32_t k1 = k0 + s.kb_split < s.kb ? k0 + s.kb_split : s.kb;
    return k1 - k0;
}

// Epilogue: a struct with
//   kChunked, kChunk               sum the k loop in chunks, of so many k-blocks
//   kStaged                        cols() uses the warp's scratch
//   kPlanes                        planes of the operands: 1, or 3 (six products a k-block)
//   Row                            what a thread keeps of its row of a tile
//   begin(tile, row, half) -> Row  row 0 .. 255 of the tile, half 0 / 1 of its columns
//   width(tile, half)              columns of the half inside the result (may be <= 0)
//   cols(Row&, c, v[32], scratch)  columns 32c .. 32c + 31 of the half (whole warps)
//   end(Row&)
template <class Epi, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_mm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Shape sh,
         const Epi epi, uint32_t* err) {
    using C = Cfg<TN>;
    constexpr uint32_t kStages = C::kStages, kStageBytes = C::kStageBytes;
    constexpr int kPlanes = Epi::kPlanes;
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2];
    __shared__ uint32_t tmem_base;
    unsigned char* ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
    const uint32_t n_tiles = sh.tm * sh.tn * sh.splits;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 16);  // 8 epilogue warps of each CTA
        }
        mbar_init_fence();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    __syncthreads();
    pair_sync();  // both CTAs run
    if (warp == 1) tmem_alloc(&tmem_base, 2 * TN);
    fence_before();
    __syncthreads();
    pair_sync();  // both hold their columns
    fence_after();
    if (warp == 1) tmem_permit_back();
    const uint32_t tmem = tmem_base;
    // a programmatic launch: set up while the kernel before finishes, and let the
    // one after do the same
    griddep_launch_dependents();
    griddep_wait();

    bool ok = true;
    if (warp == 0) {
        if (lane == 0 && !sh.stalled) {  // producer
            uint32_t it = 0;
            for (uint32_t t = pair; t < n_tiles && ok; t += n_pairs) {
                const Tile tl = tile_of(sh, t);
                const int32_t m0 = (int32_t)(tl.m * kTile + rank * kHalf), n0 = (int32_t)(tl.n * TN + rank * C::kHalfN);
                const uint32_t k0 = tl.split * sh.kb_split;
                const uint32_t k1 = k0 + sh.kb_split < sh.kb ? k0 + sh.kb_split : sh.kb;
                for (uint32_t k = k0; k < k1 && ok; ++k) {
                    const int32_t kk = (int32_t)(k * kBlockK);
                    for (int32_t p = 0; p < kPlanes; ++p, ++it) {
                        const uint32_t st = it % kStages;
                        if (it >= kStages && !wait_cluster(&empty[st], (it / kStages - 1) & 1, err, sh.wait_ns)) {
                            ok = false;
                            break;
                        }
                        if (rank == 0) mbar_arrive_tx(&full[st], 2 * kStageBytes);
                        const uint32_t bar = cluster_addr(&full[st], 0);
                        unsigned char* a = ring + st * kStageBytes;
                        unsigned char* b = a + kOperandA;
                        if (sh.a_mn) {
                            tma_load_pair(a, &map_a, m0, kk, p, bar);
                            tma_load_pair(a + kOperandA / 2, &map_a, m0 + 64, kk, p, bar);
                        } else {
                            tma_load_pair(a, &map_a, kk, m0, p, bar);
                        }
                        if (sh.b_mn) {
                            tma_load_pair(b, &map_b, n0, kk, p, bar);
                            if constexpr (TN == 256) tma_load_pair(b + 8192, &map_b, n0 + 64, kk, p, bar);
                        } else {
                            tma_load_pair(b, &map_b, kk, n0, p, bar);
                        }
                    }
                }
            }
            // the MMAs have read every stage (and every arrival on this CTA's
            // barriers has landed) before the CTA ends
            const uint32_t tail = it < kStages ? it : kStages;
            for (uint32_t i = it - tail; i < it && ok; ++i)
                ok = wait_cluster(&empty[i % kStages], (i / kStages) & 1, err, sh.wait_ns);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {  // MMA issue
            const uint32_t idesc = instr_desc(sh.a_mn, sh.b_mn, TN);
            const uint32_t step_a = sh.a_mn ? 2048 >> 4 : 32 >> 4, step_b = sh.b_mn ? 2048 >> 4 : 32 >> 4;
            uint32_t it = 0, seq = 0;
            for (uint32_t t = pair; t < n_tiles && ok; t += n_pairs) {
                const uint32_t steps = tile_steps(sh, tile_of(sh, t));
                const uint32_t chunk = Epi::kChunked ? Epi::kChunk : steps;
                for (uint32_t c0 = 0; c0 < steps && ok; c0 += chunk, ++seq) {
                    const uint32_t buf = seq & 1;
                    if (seq >= 2 && !wait_cluster(&tempty[buf], (seq / 2 - 1) & 1, err, sh.wait_ns)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t d = tmem + buf * TN;
                    const uint32_t n = steps - c0 < chunk ? steps - c0 : chunk;
                    for (uint32_t k = 0; k < n; ++k, it += kPlanes) {
                        uint64_t da[kPlanes], db[kPlanes];
#pragma unroll
                        for (uint32_t p = 0; p < (uint32_t)kPlanes; ++p) {
                            const uint32_t st = (it + p) % kStages;
                            ok = ok && wait_cluster(&full[st], ((it + p) / kStages) & 1, err, sh.wait_ns);
                            const uint32_t a = smem_u32(ring + st * kStageBytes);
                            da[p] = smem_desc(a, sh.a_mn);
                            db[p] = smem_desc(a + kOperandA, sh.b_mn);
                        }
                        if (!ok) break;
                        fence_after();
                        if constexpr (kPlanes == 1) {
#pragma unroll
                            for (uint32_t j = 0; j < kBlockK / 16; ++j)
                                mma(d, da[0] + j * step_a, db[0] + j * step_b, idesc, k > 0 || j > 0);
                        } else {
#pragma unroll
                            for (int p = 0; p < 6; ++p)
#pragma unroll
                                for (uint32_t j = 0; j < kBlockK / 16; ++j)
                                    mma(d, da[pair_a(p)] + j * step_a, db[pair_b(p)] + j * step_b, idesc,
                                        k > 0 || p > 0 || j > 0);
                        }
                        for (uint32_t p = 0; p < (uint32_t)kPlanes; ++p) commit_pair(&empty[(it + p) % kStages]);
                    }
                    if (ok) commit_pair(&tfull[buf]);
                }
            }
        }
    } else {  // epilogue: a quarter of the rows, a half of the columns a warp
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const int row = (int)rank * kHalf + quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + half * C::kHalfN;
        float* scratch = reinterpret_cast<float*>(ring + C::kRing + (warp - 2) * kScratch);  // with Epi::kStaged
        uint32_t seq = 0;
        auto wait = [&](uint32_t buf) {
            const bool good = __all_sync(0xffffffffu, wait_cluster(&tfull[buf], (seq / 2) & 1, err, sh.wait_ns));
            fence_after();
            return good;
        };
        auto done = [&](uint32_t buf) {
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(cluster_addr(&tempty[buf], 0));
        };
        // a wait that ran out: this tile's results and the next ones' are NaN
        for (uint32_t t = pair; t < n_tiles; t += n_pairs) {
            const Tile tl = tile_of(sh, t);
            const int width = epi.width(tl, half);
            if constexpr (Epi::kChunked) {
                const uint32_t chunks = (tile_steps(sh, tl) + Epi::kChunk - 1) / Epi::kChunk;
                float acc[C::kHalfN];
#pragma unroll
                for (int i = 0; i < C::kHalfN; ++i) acc[i] = 0.f;
                for (uint32_t c = 0; c < chunks && ok; ++c, ++seq) {
                    const uint32_t buf = seq & 1;
                    ok = wait(buf);
                    if (!ok) break;
#pragma unroll
                    for (int g = 0; g < C::kHalfN / 32; ++g) {
                        float v[32];
                        __syncwarp();
                        tmem_load32(lanes + buf * TN + g * 32, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[32 * g + i] += v[i];
                    }
                    done(buf);
                }
                if (!ok) {
#pragma unroll
                    for (int i = 0; i < C::kHalfN; ++i) acc[i] = __int_as_float(0x7fc00000);
                }
                typename Epi::Row r = epi.begin(tl, row, half);
#pragma unroll
                for (int g = 0; g < C::kHalfN / 32; ++g) {
                    if (g * 32 >= width) continue;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = acc[32 * g + i];
                    __syncwarp();
                    epi.cols(r, g, v, scratch);
                }
                epi.end(r);
            } else {
                const uint32_t buf = seq & 1;
                typename Epi::Row r = epi.begin(tl, row, half);
                ok = ok && wait(buf);
                for (int g = 0; g < C::kHalfN / 32 && g * 32 < width; ++g) {
                    float v[32];
                    __syncwarp();  // the load is one instruction of the whole warp
                    if (ok) {
                        tmem_load32(lanes + buf * TN + g * 32, v);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __int_as_float(0x7fc00000);
                    }
                    epi.cols(r, g, v, scratch);
                }
                epi.end(r);
                __syncwarp();
                if (ok) done(buf);
                ++seq;
            }
        }
    }
    if (!ok) {
        atomicOr(err, ERRBIT_TIMEOUT);
        // let what is in flight land before the shared memory and TMEM go
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(10000);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    pair_sync();  // the peer's arrivals on this CTA's barriers have landed
    fence_after();
    if (warp == 1) tmem_free(tmem, 2 * TN);
    __syncthreads();
    pair_sync();  // both have given their columns back
}

}  // namespace mm
}  // namespace lrs
