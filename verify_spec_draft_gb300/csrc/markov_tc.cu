// markov_tc.cu - spec_markov_grad's two products on the tcgen05 tensor cores.
//
//     WT:  dWt [V, r] = dz^T Ux     a tile of 256 entries, contraction over the rows
//     DX:  dX  [n, r] = dz Wt       a tile of 256 rows, contraction over the vocabulary
// Both run in one kernel, some pairs of CTAs on each, and go along the vocabulary together, so that
// dz is read from memory once.  A pair of CTAs
// forms a tile with cta_group::2 (M = 256, N = r up to 128 or 256): each CTA brings its 128 rows
// of A and half of B's columns, so B crosses from L2 once per pair, and the accumulator's
// two halves lie in the two CTAs' TMEM.  Per CTA, 19 warps:
//   warp 0   TMA producer: [64 x 64] boxes (128-byte swizzle) into a ring of stages.  dz is stored
//            with the vocabulary contiguous: as WT's A it is M-major, as DX's K-major, from the
//            same boxes; Ux and Wt are N-major.
//   warp 1   TMEM; in the pair's first CTA the MMA issuer
//   warp 2   (CLEAN) sets the rows without a token, whose dz may hold anything, to 0 in a stage that has
//            arrived, before it is reported to the first CTA's issuer
//   warps 3-18  epilogue: a thread owns one row and a quarter of the columns
// A tensor core's sums drop what falls below the accumulator's last bit, so a chain of steps
// ends after kMtcChunk of them: the epilogue adds it to float32 registers while the next one runs
// in the other half of TMEM.
//
// Operands are bf16.  A float32 one is split into three (bf16_parts), 24 bits in all, and the product
// is the sum of those pairs of parts that reach 2^-24 of it: 3 with one such operand, 6 with two.
// dz whose rows do not start on 16 bytes cannot be copied by TMA; it, and what is split, goes through
// a staged copy, a slice of the vocabulary at a time that stays in L2.
//
// Bound by the tensor cores: 1792 rows, V = 248,320, r = 256, bf16 take 310 us, 1.47 PFLOP/s or 75 % of the measured
// matmul rate (dz and both weights' bytes alone 190 us); the two products one after the other took 398.
// float32 operands cost their products and the staged planes: 448 rows, V = 151,936, r = 128, float32 outputs take
// 70 us in bf16, 222 with float32 weights, 334 with a float32 gradient, 536 with both.
#include "markov.cuh"
#include "tc_common.cuh"

#include <string.h>

namespace spec {

constexpr int kMtcStep = 64;                       // terms of a stage
constexpr int kMtcBox = kMtcStep * 64 * 2;         // bytes of a [64 x 64] box
constexpr int kMtcChunk = 8;                       // steps that one accumulator takes
constexpr int kMtcEpi = 16;
constexpr int kMtcThreads = 32 * (3 + kMtcEpi);

template <int NT> struct Mtc {                     // NT: columns, r rounded up to 128 or 256
    static constexpr int boxes = 2 + NT / 128;     // of a stage: A 128 x 64, B 64 x NT / 2
    static constexpr int bytes = boxes * kMtcBox;
    static constexpr int stages = NT == 256 ? 6 : 7;
    static constexpr uint32_t tmem = 2 * NT;
    static constexpr int scratch = kMtcEpi * 2048;
    static constexpr int smem = stages * bytes + scratch + 1024;
    static_assert(smem + 512 <= 227 * 1024, "shared memory");
};

// Shared-memory descriptor of an operand whose M or N runs along the 128 bytes of a swizzled row:
// 64-entry blocks a box apart (leading offset), groups of 8 terms 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(kMtcBox >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ uint32_t peer_addr(const void* p, unsigned rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
// An arrival in a CTA of the pair.  What it reports is not this thread's memory (TMEM that tcgen05.ld has waited
// for, or a stage that copies have written), so it releases nothing beyond the CTA: at cluster scope it
// would wait for the epilogue's stores (then 610 us for 284).
__device__ __forceinline__ void remote_arrive(uint64_t* bar, unsigned rank) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(peer_addr(bar, rank)) : "memory");
}
__device__ __forceinline__ bool cluster_try_wait(uint64_t* bar, unsigned parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// A wait for what either CTA of the pair does; false when it ran out.
__device__ __forceinline__ bool pair_wait(uint64_t* bar, unsigned parity, unsigned* status) {
    if (cluster_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!cluster_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            atomicOr(status, SPEC_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void umma2_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// One arrival at this barrier of `ctas` (a bit each) when every MMA issued so far completes.
__device__ __forceinline__ void umma2_commit(uint64_t* bar, unsigned short ctas = 3) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(smem_u32(bar)), "h"(ctas) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Item `it` of a pair: its tile, part and number, its steps for one pair of planes and in all.
struct MtcItem { int tile, part, number, n, all; };
// A box of a pair's CTA; `bar`, the address of a barrier of either of the two.
__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ bool mtc_item(const MarkovTc& a, int it, MtcItem& o) {
    o.number = (int)(blockIdx.x >> 1) - a.first + it * a.pairs;
    o.part = o.number / a.tiles;
    o.tile = o.number - o.part * a.tiles;
    const int blocks = (a.steps + a.block - 1) / a.block, mine = o.part < blocks ? (blocks - o.part + a.parts - 1) / a.parts : 0;
    o.n = mine * a.block - (mine > 0 && (blocks - 1) % a.parts == o.part ? blocks * a.block - a.steps : 0);
    o.all = o.n * a.terms;
    return o.part < a.parts;
}
// An item's steps in order.
struct MtcWalk {
    int at, in_block, left, term;
    __device__ __forceinline__ MtcWalk(const MarkovTc& a, const MtcItem& o) : term(0) { restart(a, o); }
    __device__ __forceinline__ void restart(const MarkovTc& a, const MtcItem& o) {
        at = o.part * a.block;
        in_block = 0;
        left = o.n;
    }
    __device__ __forceinline__ void next(const MarkovTc& a, const MtcItem& o) {
        ++at;
        if (++in_block == a.block) {
            in_block = 0;
            at += (a.parts - 1) * a.block;
        }
        if (--left == 0) {
            ++term;
            restart(a, o);
        }
    }
};

// CLEAN: WT once more, with the rows without a token as 0, where one holds what is not finite (markov_join_kernel
// finds it in dX); U's rows for them are 0, which is enough otherwise.  (Done always, by a relay of every stage, it cost 100 us of 440.)
template <int NT, bool CLEAN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMtcThreads, 1)
    markov_tc_kernel(const __grid_constant__ MarkovParams p, const __grid_constant__ MarkovBind b,
                     const __grid_constant__ MarkovTc wt, const __grid_constant__ MarkovTc dx,
                     const __grid_constant__ CUtensorMap zmap, const __grid_constant__ CUtensorMap umap,
                     const __grid_constant__ CUtensorMap wmap) {
    typedef Mtc<NT> C;
    constexpr int S = C::stages;
    extern __shared__ uint8_t mtc_raw[];
    uint8_t* ring = mtc_raw + ((1024u - (smem_u32(mtc_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t s_full[S], s_ready[S], s_empty[S], s_tfull[2], s_tempty[2], s_drain;
    __shared__ uint32_t s_tmem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = blockIdx.x & 1u;
    const bool DX = (int)(blockIdx.x >> 1) >= dx.first;
    const MarkovTc& a = DX ? dx : wt;
    pdl_launch_dependents();
    if (CLEAN) {
        pdl_wait_primary();
        if (*b.unclean == 0u) return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_ready[s], CLEAN ? 2 : 1);
            mbar_init(&s_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_tfull[s], 1);
            mbar_init(&s_tempty[s], 2 * kMtcEpi);
        }
        mbar_init(&s_drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&s_tmem)), "r"(C::tmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    pair_sync();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    MtcItem item;
    if (!CLEAN) pdl_wait_primary();   // the rows' U, what is staged, and whoever still reads dX's parts

    if (warp == 0) {
        if (lane == 0) {
            uint32_t i = 0;
            bool ok = true;
            for (int it = 0; ok && mtc_item(a, it, item); ++it) {
                const int m0 = item.tile * 256 + (int)rank * 128;
                MtcWalk walk(a, item);
                for (int k = 0; k < item.all; ++k, ++i) {
                    const uint32_t s = i % S;
                    ok = pair_wait(&s_empty[s], ((i / S) & 1u) ^ 1u, b.status);
                    if (!ok) break;
                    uint8_t* d = ring + (size_t)s * C::bytes;
                    // whom the copies report to: this CTA's warp 2, or the issuer, which expects both CTAs'
                    const uint32_t bar = CLEAN ? smem_u32(&s_full[s]) : peer_addr(&s_ready[s], 0);
                    if (CLEAN) mbar_arrive_expect_tx(&s_full[s], C::bytes);
                    else if (rank == 0) mbar_arrive_expect_tx(&s_ready[s], 2 * C::bytes);
                    const int at = walk.at * kMtcStep, za = (int)(a.planes >> (4 * walk.term)) & 3, zb = (int)(a.planes >> (4 * walk.term + 2)) & 3;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        pair_load_3d(d + j * kMtcBox, &zmap, DX ? at : m0 + 64 * j, DX ? m0 + 64 * j : at, za, bar);
#pragma unroll
                    for (int j = 0; j < NT / 128; ++j)
                        pair_load_3d(d + (2 + j) * kMtcBox, DX ? &wmap : &umap, (int)rank * (NT / 2) + j * 64, at, zb, bar);
                    walk.next(a, item);
                }
            }
            // nothing may still be on its way when the CTA ends, a copy or the issuer's arrival (which follows the
            // copies; where that did not come in time, they have had a second)
            for (uint32_t q = i > S ? i - S : 0; q < i; ++q) {
                if (CLEAN) mbar_wait(&s_full[q % S], (q / S) & 1u, b.status, kWaitLimitNs);
                ok = ok && pair_wait(&s_empty[q % S], (q / S) & 1u, b.status);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // M = 256 over the pair; B N-major, A M-major in WT
            const uint32_t idesc = idesc_bf16_f32(256, NT) | (1u << 16) | (DX ? 0u : 1u << 15);
            const uint64_t a_step = DX ? 32 / 16 : 2048 / 16;   // 16 terms on: within the swizzled rows, or 16 rows
            uint32_t i = 0, c = 0;
            bool ok = true;
            for (int it = 0; ok && mtc_item(a, it, item); ++it) {
                for (int k = 0; ok && k < item.all; ++c) {
                    const uint32_t buf = c & 1u, d = tmem + buf * NT;
                    ok = pair_wait(&s_tempty[buf], ((c >> 1) & 1u) ^ 1u, b.status);
                    const int end = min(item.all, k + kMtcChunk);
                    tc_fence_after();
                    for (bool first = true; ok && k < end; ++k, ++i, first = false) {
                        const uint32_t s = i % S;
                        ok = pair_wait(&s_ready[s], (i / S) & 1u, b.status);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t sa = smem_u32(ring + (size_t)s * C::bytes), sb = sa + 2 * kMtcBox;
                        const uint64_t da = DX ? sw128_desc(sa) : sw128_mn_desc(sa), db = sw128_mn_desc(sb);
#pragma unroll
                        for (int q = 0; q < kMtcStep / 16; ++q)
                            umma2_f16(d, da + q * a_step, db + q * (2048 / 16), idesc, first && q == 0 ? 0u : 1u);
                        umma2_commit(&s_empty[s]);
                    }
                    umma2_commit(&s_tfull[buf]);
                }
            }
            umma2_commit(&s_drain, 1);
            pair_wait(&s_drain, 0, b.status);
        }
    } else if (warp == 2) {
        uint32_t i = 0;
        bool ok = CLEAN;
        for (int it = 0; ok && mtc_item(a, it, item); ++it) {
            MtcWalk walk(a, item);
            unsigned long long marks = 0;   // a lane's step of 32
            for (int k = 0; k < item.all; ++k, ++i) {
                const uint32_t s = i % S;
                if ((walk.at & 31) == 0) marks = walk.at + lane < a.steps ? reinterpret_cast<const unsigned long long*>(b.none)[walk.at + lane] : 0;
                unsigned long long none = __shfl_sync(0xffffffffu, marks, walk.at & 31);   // rows of the step without a token
                walk.next(a, item);
                ok = mbar_wait(&s_full[s], (i / S) & 1u, b.status, kWaitLimitNs);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                if (none) {
                    uint4* z = reinterpret_cast<uint4*>(ring + (size_t)s * C::bytes);
                    for (; none; none &= none - 1) {   // a row is 8 words of each of the two boxes
                        const int row = __ffsll((long long)none) - 1;
                        if (lane < 16) z[(lane >> 3) * (kMtcBox / 16) + row * 8 + (lane & 7)] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    asm volatile("fence.acq_rel.cluster;" ::: "memory");
                    __syncwarp();
                }
                if (lane == 0) remote_arrive(&s_ready[s], 0);
            }
        }
    } else {
        constexpr int W = NT / 4;                          // columns of a thread
        const int quad = warp & 3, group = (warp - 3) >> 2;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + group * W;
        uint32_t c = 0;
        bool ok = true;
        for (int it = 0; ok && mtc_item(a, it, item); ++it) {
            float acc[W];
#pragma unroll
            for (int q = 0; q < W; ++q) acc[q] = 0.0f;
            for (int k = 0; ok && k < item.all; k += kMtcChunk, ++c) {
                const uint32_t buf = c & 1u;
                ok = pair_wait(&s_tfull[buf], (c >> 1) & 1u, b.status);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < W; q += 16) {
                    float v[16];
                    tmem_ld16(lane_base + buf * NT + q, v);
#pragma unroll
                    for (int h = 0; h < 16; ++h) acc[q + h] += v[h];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) remote_arrive(&s_tempty[buf], 0);
            }
            if (!ok) break;
            const int k0 = group * W;
            if (DX) {
                const int m = (int)rank * 128 + quad * 32 + lane;
                float* o = b.part + ((size_t)item.number * 256 + m) * NT + k0;
#pragma unroll
                for (int q = 0; q < W; q += 4) {
                    float4 x = make_float4(acc[q], acc[q + 1], acc[q + 2], acc[q + 3]);
                    if (a.add) {
                        const float4 y = *reinterpret_cast<const float4*>(o + q);
                        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                    }
                    *reinterpret_cast<float4*>(o + q) = x;
                }
            } else {
                // the thread's columns, 64 bytes at a time, through the warp's 2 KB, so that 4 lanes write
                // a row's 64 bytes (a 16-byte word a lane of 32 different rows took 284 us for 235)
                const int v0 = a.v0 + item.tile * 256 + (int)rank * 128 + quad * 32;
                uint4* sc = reinterpret_cast<uint4*>(ring + (size_t)S * C::bytes) + (warp - 3) * 128;
                const bool half = p.odt == SPEC_BF16;
                const int per = half ? 8 : 4;                  // columns of a word
#pragma unroll
                for (int q = 0; q < W; q += 16) {
                    if (half && (q & 16)) continue;
                    uint4 w[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if (half) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int at = (q + 8 * h + 2 * e) % W;
                                x[e] = pack_bf16x2(acc[at], acc[at + 1]);
                            }
                            w[h] = make_uint4(x[0], x[1], x[2], x[3]);
                        } else {
                            w[h] = make_uint4(__float_as_uint(acc[q + 4 * h]), __float_as_uint(acc[q + 4 * h + 1]),
                                              __float_as_uint(acc[q + 4 * h + 2]), __float_as_uint(acc[q + 4 * h + 3]));
                        }
                        sc[lane * 4 + (h ^ ((lane >> 1) & 3))] = w[h];
                    }
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int row = h * 8 + (lane >> 2), word = lane & 3;
                        const uint4 x = sc[row * 4 + (word ^ ((row >> 1) & 3))];
                        const int k = k0 + q + word * per;
                        if (v0 + row < a.v1 && k < p.r) {
                            const long o = (long)(v0 + row) * p.r + k;
                            if (p.r % 8 == 0) {
                                *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p.dWt_out) + o * (half ? 2 : 4)) = x;
                            } else {
                                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    if (e >= per || k + e >= p.r) break;
                                    if (half) reinterpret_cast<bf16_t*>(p.dWt_out)[o + e] = (bf16_t)(y[(e >> 1) & 3] >> (16 * (e & 1)));
                                    else reinterpret_cast<uint32_t*>(p.dWt_out)[o + e] = y[e & 3];
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
                if (CLEAN) continue;
                // dU's rows of the same entries, which lie one behind the other, as 0
                // (they start on 64 bytes, as 32 entries do; the last may end anywhere)
                const long from = (long)v0 * p.r, to = (long)min(a.v1, v0 + 32) * p.r;
                uint4* u = reinterpret_cast<uint4*>(p.dU_out);
                for (long e = from / per + group * 32 + lane; e < to / per; e += 4 * 32) u[e] = make_uint4(0u, 0u, 0u, 0u);
                const long left = to / per * per + lane;
                if (group == 0 && from < to && left < to) put(p.dU_out, p.odt, left, 0.0f);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    pair_sync();   // nobody's barriers or TMEM are in use any more
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(C::tmem) : "memory");
    }
}

// Columns [v0, v0 + columns) of dz's rows, or rows of the weights, as bf16 planes whose rows are `pitch`
// entries apart (a multiple of 8).  A thread takes 8 columns of four rows at once; bf16 rows of any
// offset are read as 16-byte words, two of them shifted into place.  Rows that `none` marks become 0.
constexpr int kStageRows = 4;
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int s) {   // from entry s of a on
    uint32_t h[9] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, 0u};
    if (s & 4)
#pragma unroll
        for (int k = 0; k < 6; ++k) h[k] = h[k + 2];
    if (s & 2)
#pragma unroll
        for (int k = 0; k < 5; ++k) h[k] = h[k + 1];
    if (s & 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = __funnelshift_r(h[k], h[k + 1], 16);
    return make_uint4(h[0], h[1], h[2], h[3]);
}
template <typename T, int PLANES>
__global__ void __launch_bounds__(256) markov_stage_kernel(const T* src, long ld, int rows, int columns, int pitch, bf16_t* out,
                                                           const uint8_t* none) {
    const int c = (int)(blockIdx.x * blockDim.x + threadIdx.x) * 8;
    pdl_launch_dependents();
    if (c >= columns) return;
    const int step = (int)(gridDim.y * blockDim.y);
    const bool inside = c >= 8 && c + 16 <= columns;   // every word that is touched lies in the row
    for (int row0 = (int)(blockIdx.y * blockDim.y + threadIdx.y); row0 < rows; row0 += kStageRows * step) {
        if constexpr (sizeof(T) == 2) {
            uint4 a[kStageRows], b[kStageRows];
            int mis[kStageRows];
#pragma unroll
            for (int q = 0; q < kStageRows; ++q) {
                const int row = min(row0 + q * step, rows - 1);
                const T* from = src + row * ld;
                mis[q] = (int)((reinterpret_cast<uintptr_t>(from) & 15u) / 2u);
                if (inside) {
                    const uint4* w = reinterpret_cast<const uint4*>(from - mis[q] + c);
                    a[q] = __ldg(w);
                    b[q] = __ldg(w + 1);
                }
            }
            pdl_wait_primary();   // the marks, and whoever still reads the last slice
#pragma unroll
            for (int q = 0; q < kStageRows; ++q) {
                const int row = row0 + q * step;
                if (row >= rows) continue;
                if (!inside) {
                    const RowWords<T> in(src + row * ld, columns);
                    a[q] = in.load(c / 8);
                    if (in.mis && c / 8 + 1 < in.n) b[q] = in.load(c / 8 + 1);
                    else b[q] = make_uint4(0u, 0u, 0u, 0u);
                }
                const bool off = none && (none[row >> 3] >> (row & 7)) & 1;
                *reinterpret_cast<uint4*>(out + (long)row * pitch + c) = off ? make_uint4(0u, 0u, 0u, 0u) : shifted(a[q], b[q], mis[q]);
            }
        } else {
            float x[kStageRows][8];
#pragma unroll
            for (int q = 0; q < kStageRows; ++q) {
                const T* from = src + min(row0 + q * step, rows - 1) * ld + c;
                if (inside && (reinterpret_cast<uintptr_t>(from) & 15u) == 0) {
                    const float4 a = __ldg(reinterpret_cast<const float4*>(from)), b = __ldg(reinterpret_cast<const float4*>(from) + 1);
                    x[q][0] = a.x; x[q][1] = a.y; x[q][2] = a.z; x[q][3] = a.w;
                    x[q][4] = b.x; x[q][5] = b.y; x[q][6] = b.z; x[q][7] = b.w;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[q][k] = c + k < columns ? load_one(from + k) : 0.0f;
                }
            }
            pdl_wait_primary();
#pragma unroll
            for (int q = 0; q < kStageRows; ++q) {
                const int row = row0 + q * step;
                if (row >= rows) continue;
                float y[8][3];
                const bool off = none && (none[row >> 3] >> (row & 7)) & 1;
#pragma unroll
                for (int k = 0; k < 8; ++k) bf16_parts(off ? 0.0f : x[q][k], y[k]);
#pragma unroll
                for (int h = 0; h < PLANES; ++h) {
                    const float z[8] = {y[0][h], y[1][h], y[2][h], y[3][h], y[4][h], y[5][h], y[6][h], y[7][h]};
                    *reinterpret_cast<uint4*>(out + ((long)h * rows + row) * pitch + c) = word_of<bf16_t>(z);
                }
            }
        }
    }
}
static cudaError_t mtc_stage(const void* src, int dtype, long at, long ld, int rows, int columns, int pitch, bf16_t* out,
                      const uint8_t* none, cudaStream_t stream) {
    const dim3 block = columns <= 256 ? dim3(32, 8) : dim3(256, 1);   // a thread per 8 columns, 4 rows each
    const unsigned x = (unsigned)((columns + 8 * block.x - 1) / (8 * block.x)), y = (unsigned)((rows + kStageRows * block.y - 1) / (kStageRows * block.y));
    const dim3 grid(x, y < 65535u ? y : 65535u);
    if (dtype == SPEC_BF16)
        return launch_behind(markov_stage_kernel<bf16_t, 1>, grid, block, 0, stream, reinterpret_cast<const bf16_t*>(src) + at, ld, rows, columns, pitch, out, none);
    return launch_behind(markov_stage_kernel<float, 3>, grid, block, 0, stream, reinterpret_cast<const float*>(src) + at, ld, rows, columns, pitch, out, none);
}

static bool mtc_map(CUtensorMap* m, const void* base, int width, long rows, long pitch, int planes) {
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)pitch * 2 * (cuuint64_t)rows};
    const cuuint32_t box[3] = {64, 64, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    EncodeTiledFn f = encode_tiled();
    return f && f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The pairs of each product and dX's parts: the fewest steps in a line, over the parts and the rounds that
// dX's items take on its pairs.  A tile of dWt takes its steps, or the time its rows and dU's take to be written
// (8 steps for 256 x 256 float32 of both); an item's start and end count as 12 steps, a part's share of the join
// as half a one.  A part takes blocks of as many steps as dWt's pairs pass meanwhile.
static void mtc_plan(int n, int columns, int r, int out_size, int terms, int pairs, MarkovTc& wt, MarkovTc& dx) {
    memset(&wt, 0, sizeof(wt));
    memset(&dx, 0, sizeof(dx));
    wt.tiles = (columns + 255) / 256;
    wt.steps = wt.block = (n + kMtcStep - 1) / kMtcStep;
    wt.parts = 1;
    dx.tiles = (n + 255) / 256;
    dx.steps = (columns + kMtcStep - 1) / kMtcStep;
    wt.terms = dx.terms = terms;
    double best = -1.0;
    const double written = 8.0 * r * out_size / 1024.0;
    // (more tiles than parts are cut for: as many rounds as leave dWt its share; 65,536 rows, V = 32,000, r = 64
    // take 1.4 ms, 3.9 with four)
    const int most_rounds = dx.tiles > kMarkovItems ? 64 : 4;
    for (int parts = 1; parts <= dx.steps && (parts == 1 || parts * dx.tiles <= kMarkovItems); ++parts)
        for (int rounds = 1; rounds <= most_rounds; ++rounds) {
            const int items = parts * dx.tiles, dp = (items + rounds - 1) / rounds, wp = pairs - dp;
            if (wp < 1 || (rounds > 1 && dp == (items + rounds - 2) / (rounds - 1))) continue;
            const double tile = wt.steps * terms > written ? wt.steps * terms : written;
            const double w = (double)((wt.tiles + wp - 1) / wp) * (tile + 1.0) + 12.0;
            const double d = rounds * ((double)((dx.steps + parts - 1) / parts) * terms + 12.0);
            const double cost = (w > d ? w : d) + 0.5 * items;
            if (best < 0.0 || cost < best) {
                best = cost;
                dx.parts = parts;
                dx.pairs = dp;
            }
        }
    if (best < 0.0) {   // more tiles than the rounds take on a smaller device
        dx.parts = 1;
        dx.pairs = pairs / 2;
    }
    const int left = pairs - dx.pairs;
    wt.first = 0;
    wt.pairs = wt.tiles < left ? wt.tiles : left;
    dx.first = wt.pairs;
    const int pass = 4 * wt.pairs / dx.parts < 1 ? 1 : 4 * wt.pairs / dx.parts;   // (256 entries are 4 steps)
    const int share = (dx.steps + dx.parts - 1) / dx.parts, blocks = (share + pass / 2) / pass < 1 ? 1 : (share + pass / 2) / pass;
    dx.block = (share + blocks - 1) / blocks;
}

template <int NT>
static cudaError_t mtc_launch(const MarkovParams& p, const MarkovBind& b, cudaStream_t stream) {
    const int n = p.B * p.gamma, r8 = round8(p.r);
    const bool z16 = p.gdt == SPEC_BF16, w16 = p.wdt == SPEC_BF16;
    const bool stage_z = !z16 || p.ld % 8 != 0, stage_w = !w16 || p.r != r8;
    // as many columns as the stage takes of what is staged
    const size_t each = 2 * ((stage_z ? (size_t)n * (z16 ? 1 : 3) : 0) + (stage_w ? (size_t)r8 * (w16 ? 1 : 3) : 0));
    const size_t room = each ? (b.stage_bytes - 512) / each : 0;
    const int columns = each && room < (size_t)round8(p.V) ? (int)(room / 256 * 256) : p.V;
    bf16_t* zs = b.stage;
    bf16_t* ws = b.stage + (stage_z ? (align256((size_t)n * (z16 ? 1 : 3) * round8(columns) * 2) / 2) : 0);
    const int pairs = device_sm_count() / 2 > kMarkovPairs ? kMarkovPairs : (device_sm_count() / 2 > 2 ? device_sm_count() / 2 : 2);
    const int terms = z16 ? (w16 ? 1 : 3) : (w16 ? 3 : 6);
    // (A's part, B's part) of each term, the smallest products first
    const unsigned planes = z16 ? (w16 ? 0u : 0x048u) : (w16 ? 0x012u : 0x041528u);
    MarkovTc wt, dx;
    mtc_plan(n, columns, p.r, p.odt == SPEC_BF16 ? 2 : 4, terms, pairs, wt, dx);
    wt.planes = dx.planes = planes;
    auto kern = markov_tc_kernel<NT, false>;
    auto clean = markov_tc_kernel<NT, true>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Mtc<NT>::smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(clean, cudaFuncAttributeMaxDynamicSharedMemorySize, Mtc<NT>::smem);
    if (e != cudaSuccess) return e;
    CUtensorMap zmap, umap, wmap;
    if (!mtc_map(&umap, b.ux, p.r, n, r8, w16 ? 1 : 3)) return cudaErrorInvalidValue;
    for (int v0 = 0; v0 < p.V; v0 += columns) {
        const int width = columns < p.V - v0 ? columns : p.V - v0;
        if (stage_z) e = mtc_stage(p.grad, p.gdt, v0, p.ld, n, width, round8(width), zs, b.none, stream);
        if (stage_w && e == cudaSuccess) e = mtc_stage(p.Wt, p.wdt, (long)v0 * p.r, p.r, width, p.r, r8, ws, nullptr, stream);
        if (e != cudaSuccess) return e;
        if (!mtc_map(&zmap, stage_z ? zs : reinterpret_cast<const bf16_t*>(p.grad) + v0, width, n, stage_z ? round8(width) : p.ld, z16 ? 1 : 3) ||
            !mtc_map(&wmap, stage_w ? ws : reinterpret_cast<const bf16_t*>(p.Wt) + (long)v0 * p.r, p.r, width, r8, w16 ? 1 : 3))
            return cudaErrorInvalidValue;
        wt.tiles = (width + 255) / 256;
        dx.steps = (width + kMtcStep - 1) / kMtcStep;
        wt.v0 = dx.v0 = v0;
        wt.v1 = dx.v1 = v0 + width;
        dx.add = v0 > 0;
        e = launch_behind(kern, dim3(2u * (unsigned)(wt.pairs + dx.pairs)), kMtcThreads, Mtc<NT>::smem, stream, p, b, wt, dx, zmap, umap, wmap);
        if (e != cudaSuccess) return e;
    }
    e = markov_join(p, b, {dx.parts, (long)dx.tiles * 256, NT}, stream);
    if (e != cudaSuccess) return e;
    if (!stage_z) {   // (a staged row without a token is 0)
        if (!mtc_map(&zmap, p.grad, p.V, n, p.ld, 1)) return cudaErrorInvalidValue;
        wt.tiles = (p.V + 255) / 256;
        wt.v0 = 0;
        wt.v1 = p.V;
        wt.pairs = dx.first = wt.tiles < pairs ? wt.tiles : pairs;
        e = launch_behind(clean, dim3(2u * (unsigned)wt.pairs), kMtcThreads, Mtc<NT>::smem, stream, p, b, wt, dx, zmap, umap, umap);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t markov_tc_launch(const MarkovParams& p, const MarkovBind& b, cudaStream_t stream) {
    return p.r > 128 ? mtc_launch<256>(p, b, stream) : mtc_launch<128>(p, b, stream);
}

}  // namespace spec
