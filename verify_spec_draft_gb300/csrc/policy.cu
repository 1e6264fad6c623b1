// policy.cu - the clipped policy loss of sampled tokens (spec_policy_loss) and its gradient.
//
// With q = softmax(z / t), lp = ln q_x, u = exp(lp - old), d = ref - lp:
//     L       = -min(u A, clip(u) A) + kl (e^d - d - 1)
//     dL/dz_v = (slope / t) ([v = x] - q_v),  slope = dL/dlp
// The slope is one number per row, known once the row's maximum and sum are, so a row is read
// once: a cluster of CTAs shares it, each CTA keeps its slice in shared memory between the
// statistics and the gradient, and the CTAs meet once, by (maximum, sum) pairs written into one
// another's shared memory.  1 - q_x is summed over the other entries, so a token of probability
// near 1 keeps its gradient's digits.
// Bound by memory: a row in, its gradient out (1792 rows of 248,320 bf16, one in ten of weight 0: 285 us,
// 88 % of the measured copy rate in what moves; 448 rows' loss alone, where one in ten is not read either: 37 us,
// 81 %; all 448 read: 36.5 us, 91 %, in float32 68 us, 98 %).
#include "internal.h"
#include "row_words.cuh"

#include <type_traits>

namespace spec {

constexpr int kPolThreads(int mode) { return mode == 0 ? 128 : 256; }
constexpr int kPolBatch(int mode) { return mode == 1 ? 4 : 8; }   // words a thread takes at once
constexpr int kPolChunks = 4;                      // copies of a slice
constexpr int kPolMaxCluster = 16;
constexpr int kPolMost = 220 * 1024;               // bytes of a slice that can be kept
constexpr int kPolSlice = 3392;                    // words of one that is kept where the rows are many

// Pairs (m, s): the maximum of some entries and the sum of their weights relative to it
// (row_words.cuh); empty: (-inf, 0).  NaN shows in m.
__device__ __forceinline__ float pol_weight(float2 v, float m, float c) {
    return v.x == -INFINITY ? 0.0f : v.y * ex2(ref_rel(v.x, m, c));
}
__device__ __forceinline__ float2 pol_merge(float2 a, float2 b, float c) {
    const float m = f_max_nan(a.x, b.x);
    return make_float2(m, pol_weight(a, m, c) + pol_weight(b, m, c));
}
// log2 of what a sum relative to R(a) is worth relative to R(b): both products rounded as the sums'
// were, which a fused multiply-add would undo (3e5 from zero that cost lp 1e-4)
__device__ __forceinline__ float pol_step(float a, float b, float c) {
    const float x = __fmul_rn(a, c), y = __fmul_rn(b, c);
    return ref_near(x) && ref_near(y) ? __fsub_rn(x, y) : ref_step_far(a, b, c);
}

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A pair into the place `here` of CTA `rank`, whose barrier `bar` counts its 8 bytes.  (A cluster barrier
// with release would wait for all of the last row's gradient to be written first.)
__device__ __forceinline__ void cluster_put(float2* here, uint64_t* bar, unsigned rank, float2 v) {
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(here)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];"
                 :: "r"(a), "f"(v.x), "f"(v.y), "r"(b) : "memory");
}

// A wait of 1 s at most, or of the workspace's patience (us, 1000 at least) where that is not 0.
__device__ __forceinline__ bool pol_wait(uint64_t* bar, unsigned parity, const PolicyParams& p) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        const unsigned long long waited = global_timer_ns() - t0;
        if (waited < 1000000ull) continue;
        const unsigned us = *(const volatile unsigned*)&p.wait->patience;
        if (waited > (us ? us * 1000ull : kWaitLimitNs)) {
            atomicOr(p.status, SPEC_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}

// What the row's CTAs make of its statistics (each for itself).
struct PolRow {
    float loss, lp;
    float ref, m, factor;   // gradient of entry v: -2^(z c - ref) factor; beyond kRefNear -2^((z - m) c) factor
    float at_token;         // gradient of x
    int bad, slope_bad;
};
// The row's own numbers; zx: x's logit
struct PolInputs { float old, A, ref, wt, zx; bool token_ok; };
// T: the pair of the entries but x
__device__ __forceinline__ PolRow policy_row(const PolicyParams& p, float2 T, const PolInputs& in) {
    PolRow r;
    const float c = p.scale;
    const float old = in.old, A = in.A, ref = in.ref, wt = in.wt, zx = in.zx;
    const float2 A2 = pol_merge(T, make_float2(zx, zx == -INFINITY ? 0.0f : 1.0f), c);
    const float M = A2.x, Z = A2.y;
    r.bad = !in.token_ok || !(M < INFINITY) || M == -INFINITY || !(fabsf(old) < INFINITY) || !(fabsf(A) < INFINITY) ||
            !(fabsf(ref) < INFINITY) || !(fabsf(wt) < INFINITY);
    // the difference before the scaling: lp keeps its digits whatever the row's offset
    const float lp = zx == -INFINITY ? -INFINITY : fmaf(zx - M, p.inv_t, -logf(Z));
    const float u = expf(lp - old);
    float loss = 0.0f, slope = 0.0f;
    if (A != 0.0f) {
        loss = -fminf(u * A, fminf(fmaxf(u, p.low), p.high) * A);
        if (A > 0.0f ? u <= p.high : u >= p.low) slope = -u * A;
    }
    if (p.ref_logp) {
        const float d = ref - lp, e = expm1f(d);
        loss += d < INFINITY ? p.kl * (e - d) : INFINITY;
        slope -= p.kl * e;
    }
    r.lp = lp;
    r.loss = loss;
    const float k = slope * (wt * p.inv_t);
    r.slope_bad = !(fabsf(slope) < INFINITY && fabsf(k) < INFINITY);
    r.m = M;
    r.ref = M * c;
    r.factor = k / Z * ref_fix(M, c);
    r.at_token = k * (pol_weight(T, M, c) / Z);
    if (r.bad) r.loss = r.lp = NAN;
    if (r.bad || r.slope_bad) r.factor = r.at_token = NAN;
    return r;
}

// MODE: 0 the loss alone; 1 with the gradient, the slice kept in shared memory; 2 with the gradient,
// the slice read again (it is too large to keep).  A cluster takes one row in n_clusters; in MODE 1 the
// next row's slice is on its way as soon as every thread has read the last of this one's.
template <typename T, int MODE, bool ALIGNED>
__global__ void __launch_bounds__(kPolThreads(MODE), MODE == 0 ? 6 : 4) policy_kernel(const __grid_constant__ PolicyParams p) {
    constexpr int E = 16 / (int)sizeof(T), TH = kPolThreads(MODE), WARPS = TH / 32, BATCH = kPolBatch(MODE);
    extern __shared__ __align__(128) uint8_t s_slice[];
    __shared__ __align__(8) uint64_t s_full[kPolChunks], s_met[2];
    __shared__ float2 s_pair[2][kPolMaxCluster], s_warp[WARPS];
    __shared__ PolRow s_row;
    __shared__ int s_gone;          // a wait of this CTA has run out
    __shared__ unsigned s_withheld;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = cluster_rank(), size = cluster_size();
    const int n_clusters = (int)(gridDim.x / size);
    const float c = p.scale;
    uint4* slot = reinterpret_cast<uint4*>(s_slice);
    if (tid == 0) {
        for (int q = 0; q < kPolChunks; ++q) mbar_init(&s_full[q], 1);
        for (int q = 0; q < 2; ++q) mbar_init(&s_met[q], 1);
        s_gone = 0;
        s_withheld = 0u;
        fence_mbar_init();
    }
    __syncthreads();
    cluster_arrive();   // so that no CTA writes into one that has not begun
    if (tid == 96 && blockIdx.x == 0) s_withheld = *(const volatile unsigned*)&p.wait->withheld;
    // a row's slice: words [first, first + n) of the row, whole words [a, b) of those
    auto row_of = [&](int row) { return SegWords<T, ALIGNED>(reinterpret_cast<const T*>(p.logits) + (long)row * p.ld, p.V); };
    const int first = (int)rank * p.slice;
    auto words_of = [&](const SegWords<T, ALIGNED>& in) { return max(0, min(in.n() - first, p.slice)); };
    // words of a copy: whole batches
    auto per_of = [&](int n) { return (n + kPolChunks * TH * BATCH - 1) / (kPolChunks * TH * BATCH) * (TH * BATCH); };
    auto weight_of = [&](int row) { return row < p.rows ? (p.weight ? p.weight[row] : 1.0f) : 0.0f; };
    auto issue = [&](int row) {   // (all threads; the slot is free)
        const SegWords<T, ALIGNED> in = row_of(row);
        const int n = words_of(in), per = per_of(n);
        const int a = !ALIGNED && n > 0 && !in.r.whole(first) ? 1 : 0;
        const int b = !ALIGNED && n > a && !in.r.whole(first + n - 1) ? n - 1 : max(n, a);
        if (tid == 0) {
            for (int q = 0; q < kPolChunks; ++q) {
                const int lo = max(a, q * per), hi = min(b, (q + 1) * per);
                if (lo < hi) {
                    mbar_arrive_expect_tx(&s_full[q], (unsigned)(hi - lo) * 16u);
                    bulk_g2s(slot + lo, in.r.p + in.entry(first + lo), (unsigned)(hi - lo) * 16u, &s_full[q]);
                } else {
                    mbar_arrive1(&s_full[q]);
                }
            }
        } else if (tid == 32 && a > 0) {
            slot[0] = in.load(first);
        } else if (tid == 64 && b < n) {
            slot[b] = in.load(first + b);
        }
    };
    // Warp 0: this CTA's pair to all of the cluster's, and v becomes all of theirs together; false when one
    // did not come in time.  Places are used in turn: the pairs of row i + 2 come after every CTA's of row
    // i + 1, which it sends when it has read those of row i.  (A CTA that has waited in vain meets no more: its
    // barrier's phase is still open, and may not be armed again.)
    auto meet = [&](int i, float2& v) {
        float2* pairs = s_pair[i & 1];
        uint64_t* bar = &s_met[i & 1];
        if (lane < (MODE == 0 ? 1 : (int)size) && s_withheld != (unsigned)i + 1u) cluster_put(&pairs[rank], bar, lane, v);
        if (MODE == 0 && rank != 0) return true;   // (for the first CTA alone)
        if (lane == 0) mbar_arrive_expect_tx(bar, size * 8u);
        const bool here = __all_sync(0xffffffffu, pol_wait(bar, (i >> 1) & 1, p));
        v = lane < (int)size ? pairs[lane] : make_float2(-INFINITY, 0.0f);
        const float m = warp_max_nan(v.x);
        v = make_float2(m, warp_sum(pol_weight(v, m, c)));
        return here;
    };
    int row = (int)(blockIdx.x / size);
    float wt = weight_of(row);
    if (MODE == 1 && wt != 0.0f) issue(row);
    bool begun = false;
    int live = 0, copies = 0;   // rows that counted so far, and those whose copies were waited for
    int lost = -1;              // (warp 0) the meeting that one of the cluster did not come to in time
    for (; row < p.rows; row += n_clusters) {
        const SegWords<T, ALIGNED> in = row_of(row);
        T* d = reinterpret_cast<T*>(p.grad_out) + (long)row * p.ld;
        const int n = words_of(in), next = row + n_clusters;
        const float next_wt = weight_of(next);
        if (wt == 0.0f) {
            if (MODE)
                for (int l = tid; l < n; l += TH) in.store(d, first + l, make_uint4(0u, 0u, 0u, 0u));
            if (rank == 0 && tid == 0) p.loss_out[row] = p.logp_out[row] = 0.0f;
            if (MODE == 1 && next_wt != 0.0f) issue(next);   // nothing is in the slot
            wt = next_wt;
            continue;
        }
        const int x = p.tokens[row];
        const bool token_ok = x >= 0 && x < p.V;
        PolInputs mine = {0.0f, 0.0f, 0.0f, wt, -INFINITY, token_ok};
        if (tid == 0) {
            mine.old = p.old_logp[row];
            mine.A = p.advantage[row];
            if (p.ref_logp) mine.ref = p.ref_logp[row];
            // before any CTA writes, as the gradient may replace the row
            if (token_ok) {
                const T* z = in.r.p + x;
                if (sizeof(T) == 2) mine.zx = to_float((bf16_t)*reinterpret_cast<const volatile unsigned short*>(z));
                else mine.zx = to_float(*reinterpret_cast<const volatile float*>(z));
            }
        }
        const int xe = token_ok ? x + (ALIGNED ? 0 : in.r.mis) : -1;
        const int xl = token_ok ? xe / E - first : -1;      // x's word in the slice (or outside it)
        const uint32_t xbit = token_ok ? 1u << (xe % E) : 0u;
        __syncthreads();   // (the words that are not whole)

        float m = -INFINITY, s = 0.0f;
        // words [l0, end): whole batches of all threads, then one by one
        auto take = [&](auto count, const uint4* w, float& m, float& s) {
            constexpr int N = decltype(count)::value;
            float bm = m;
#pragma unroll
            for (int q = 0; q < N; ++q) bm = f_max_nan(bm, u4_max_nan<sizeof(T)>(w[q]));
            if (bm != m) {
                s = m == -INFINITY ? 0.0f : s * ex2(pol_step(m, bm, c));
                m = bm;
            }
            uint4 v[N];
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] = w[q];
            s += words_sum<T, N>(v, m, c);
        };
        auto word = [&](int l) {
            uint4 w = MODE == 1 ? slot[l] : in.load(first + l);
            if (l == xl) w = word_without<T>(w, xbit);
            return w;
        };
        auto batch = [&](int l0, int end) {
            for (; l0 + TH * BATCH <= end; l0 += TH * BATCH) {
                uint4 w[BATCH];
#pragma unroll
                for (int q = 0; q < BATCH; ++q) w[q] = word(l0 + q * TH + tid);
                take(std::integral_constant<int, BATCH>(), w, m, s);
            }
#pragma unroll 1
            for (int l = l0 + tid; l < end; l += TH) {
                const uint4 w[1] = {word(l)};
                take(std::integral_constant<int, 1>(), w, m, s);
            }
        };
        bool late = false;
        if (MODE == 1) {
            const int per = per_of(n);
            for (int q = 0; q < kPolChunks; ++q) {
                late |= !pol_wait(&s_full[q], copies & 1, p);
                const int end = min(n, (q + 1) * per);
                if (!late) batch(q * per, end);
            }
            ++copies;
            if (late) s_gone = 1;
        } else {
            batch(0, n);
        }
        if (late) m = NAN;
        {
            float2 v = make_float2(m, s * ref_fix(m, c));
            const float wm = warp_max_nan(v.x);
            v = make_float2(wm, warp_sum(pol_weight(v, wm, c)));
            if (lane == 0) s_warp[warp] = v;
        }
        __syncthreads();
        if (!begun) cluster_wait();
        begun = true;
        if (warp == 0) {
            float2 v = lane < WARPS ? s_warp[lane] : make_float2(-INFINITY, 0.0f);
            const float wm = warp_max_nan(v.x);
            v = make_float2(wm, warp_sum(pol_weight(v, wm, c)));
            // x's logit is here before the other CTAs learn of the pair, and may write over it
            mine.zx = __shfl_sync(0xffffffffu, mine.zx, 0);
            if (!meet(live, v)) {
                v.x = NAN;
                lost = live;
                if (lane == 0) s_gone = 1;
            }
            if (lane == 0 && (MODE || rank == 0)) {
                const PolRow r = policy_row(p, v, mine);
                s_row = r;
                if (rank == 0) {
                    p.loss_out[row] = r.loss;
                    p.logp_out[row] = r.lp;
                    if (!token_ok) atomicOr(p.status, SPEC_DEV_TOKEN);
                    else if (r.bad || (MODE && r.slope_bad)) atomicOr(p.status, SPEC_DEV_NONFINITE);
                }
            }
        }
        ++live;
        wt = next_wt;
        if (!MODE) continue;
        __syncthreads();
        const PolRow r = s_row;
        const float f = -r.factor;
        const bool near = ref_near(r.ref);
        const f2x cc = f2_pack(c, c), mm = f2_pack(-r.ref, -r.ref), ff = f2_pack(f, f);
#pragma unroll 4
        for (int l = tid; l < n; l += TH) {
            const uint4 w = MODE == 1 ? slot[l] : in.load(first + l);
            float g[E];
            if (near) {
#pragma unroll
                for (int k = 0; k < E; k += 2) {
                    const float2 y = f2_unpack(f2_mul(
                        f2_ex2(f2_fma(f2_pack(word_entry<T>(w, k), word_entry<T>(w, k + 1)), cc, mm)), ff));
                    g[k] = y.x;
                    g[k + 1] = y.y;
                }
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) g[k] = ex2((word_entry<T>(w, k) - r.m) * c) * f;
            }
            if (l == xl) {
#pragma unroll
                for (int k = 0; k < E; ++k) g[k] = (xbit >> k) & 1u ? r.at_token : g[k];
            }
            in.store(d, first + l, word_of<T>(g));
        }
        if (MODE == 1 && !ALIGNED) fence_proxy_async_smem();   // words written here, before the copy that may cover them
        __syncthreads();   // the slot has been read, and s_row and s_warp
        if (MODE == 1) {
            if (s_gone) break;   // (the same for every thread)
            if (next_wt != 0.0f) issue(next);
        }
    }
    if (!begun) cluster_wait();
    if (MODE == 1 && row < p.rows) {
        // a copy or a pair has not come in time: nothing of this CTA's may still be on its way when it ends, and the
        // rest of its rows' slices have no gradient.  The cluster's other CTAs wait for its next pair in vain, and
        // do the same.
        for (int q = 0; q < kPolChunks; ++q) pol_wait(&s_full[q], (copies - 1) & 1, p);
        for (row += n_clusters; row < p.rows; row += n_clusters) {
            const SegWords<T, ALIGNED> in = row_of(row);
            const uint32_t nan = sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu;
            const bool on = weight_of(row) != 0.0f;
            T* d = reinterpret_cast<T*>(p.grad_out) + (long)row * p.ld;
            for (int l = tid, n = words_of(in); l < n; l += TH)
                in.store(d, first + l, on ? make_uint4(nan, nan, nan, nan) : make_uint4(0u, 0u, 0u, 0u));
            if (rank == 0 && tid == 0) p.loss_out[row] = p.logp_out[row] = on ? NAN : 0.0f;
        }
    }
    // a CTA's memory stays until the last pair that was sent to it is in (the loss alone: the first CTA's)
    cluster_arrive();
    if (MODE || rank == 0) cluster_wait();
    // (one that was late may still be on its way)
    if (warp == 0 && lost >= 0)
        for (const unsigned long long t0 = global_timer_ns();
             !mbar_try_wait(&s_met[lost & 1], (lost >> 1) & 1) && global_timer_ns() - t0 < 1000000ull;) {}
}

// The cluster's size.  With the gradient: slices of 53 KB at most, so that four CTAs share an SM and some load
// while others form their gradient (1792 rows of 248,320 bf16: ten CTAs of 50 KB 285 us; before the sums
// took whole batches 299, with eight of 62 KB and three an SM 314, with more and smaller ones 338 and up, as the
// registers hold four).
// The loss alone keeps nothing, so a CTA takes a whole row where the rows are enough to fill the
// device (448 rows: two CTAs a row 38 us, eight 40).  More CTAs per row where the rows are few, down to
// a batch of words per thread.
template <typename T>
static cudaError_t policy_typed(PolicyParams p, cudaStream_t stream) {
    constexpr int E = 16 / (int)sizeof(T);
    const int words = (p.V + 2 * E - 2) / E;   // whatever the row's offset
    const int sms = device_sm_count();
    int size = 1;
    if (p.grad_out) {
        size = (words + kPolSlice - 1) / kPolSlice;
        if (size > kPolMaxCluster) size = kPolMaxCluster;
        while (size <= 4 && (long)p.rows * size < sms && words / (2 * size) >= 256) size *= 2;
    } else {
        while (size < kPolMaxCluster && (long)p.rows * size < 5 * sms && words / (2 * size) >= 512) size *= 2;
    }
    p.slice = (words + size - 1) / size;
    const size_t bytes = (size_t)p.slice * 16;
    const int mode = !p.grad_out ? 0 : (bytes <= kPolMost ? 1 : 2);
    const bool fits = SegWords<T, true>::fits(p.ld, p.V);
    const void* kerns[3][2] = {{(const void*)policy_kernel<T, 0, false>, (const void*)policy_kernel<T, 0, true>},
                               {(const void*)policy_kernel<T, 1, false>, (const void*)policy_kernel<T, 1, true>},
                               {(const void*)policy_kernel<T, 2, false>, (const void*)policy_kernel<T, 2, true>}};
    const void* kern = kerns[mode][fits];
    cudaError_t e = cudaSuccess;
    if (size > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    // (always: what a launch gets without it, 48 KB, is for the slice and the kernel's own arrays together)
    if (e == cudaSuccess && mode == 1) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPolMost);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3((unsigned)kPolThreads(mode));
    cfg.dynamicSmemBytes = mode == 1 ? bytes : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = p.rows;
    if (mode == 1 && (long)p.rows * size > 2 * sms) {
        // as many as the device holds at once (the rest would wait for a whole share of the rows)
        int most = 0;
        cfg.gridDim = dim3((unsigned)size);
        e = cudaOccupancyMaxActiveClusters(&most, kern, &cfg);
        if (e != cudaSuccess) return e;
        if (most < 1) return cudaErrorInvalidConfiguration;
        if (clusters > most) clusters = most;
    }
    cfg.gridDim = dim3((unsigned)clusters * (unsigned)size);
    void* args[] = {&p};
    e = cudaLaunchKernelExC(&cfg, kern, args);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t policy_launch(PolicyParams p, cudaStream_t stream) {
    return p.dtype == SPEC_BF16 ? policy_typed<bf16_t>(p, stream) : policy_typed<float>(p, stream);
}

}  // namespace spec
