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
#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kPolThreads = 256;
constexpr int kPolWarps = kPolThreads / 32;
constexpr int kPolBatch = 4;                       // words a thread takes at once
constexpr int kPolChunks = 4;                      // copies of a slice
constexpr int kPolMaxCluster = 16;

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
__device__ __forceinline__ void cluster_put(float2* here, unsigned rank, float2 v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(here)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" :: "r"(a), "f"(v.x), "f"(v.y) : "memory");
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
// the slice read again (it is too large to keep)
template <typename T, int MODE>
__global__ void __launch_bounds__(kPolThreads) policy_kernel(const __grid_constant__ PolicyParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) uint8_t s_slice[];
    __shared__ __align__(8) uint64_t s_full[kPolChunks];
    __shared__ float2 s_pair[kPolMaxCluster], s_warp[kPolWarps];
    __shared__ PolRow s_row;
    __shared__ int s_late;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = cluster_rank(), size = cluster_size();
    const int row = (int)(blockIdx.x / size);
    const float c = p.scale;
    cluster_arrive();   // so that no CTA writes into one that has not begun
    const float wt = p.weight ? p.weight[row] : 1.0f;
    const T* z = reinterpret_cast<const T*>(p.logits) + (long)row * p.ld;
    T* d = reinterpret_cast<T*>(p.grad_out) + (long)row * p.ld;
    const RowWords<T> in(z, p.V);
    const int first = (int)rank * p.slice, n = max(0, min(in.n - first, p.slice));
    if (wt == 0.0f) {
        cluster_wait();
        if (MODE)
            for (int l = tid; l < n; l += kPolThreads) in.store(d, first + l, make_uint4(0u, 0u, 0u, 0u));
        if (rank == 0 && tid == 0) p.loss_out[row] = p.logp_out[row] = 0.0f;
        return;
    }
    // whole words [a, b) of the slice
    const int a = n > 0 && !in.whole(first) ? 1 : 0;
    const int b = n > a && !in.whole(first + n - 1) ? n - 1 : max(n, a);
    uint4* slot = reinterpret_cast<uint4*>(s_slice);
    const int per = ((n + kPolChunks - 1) / kPolChunks + 7) & ~7;   // words of a copy
    if (MODE == 1) {
        if (tid == 0) {
            for (int q = 0; q < kPolChunks; ++q) mbar_init(&s_full[q], 1);
            s_late = 0;
            fence_mbar_init();
            for (int q = 0; q < kPolChunks; ++q) {
                const int lo = max(a, q * per), hi = min(b, (q + 1) * per);
                if (lo < hi) {
                    mbar_arrive_expect_tx(&s_full[q], (unsigned)(hi - lo) * 16u);
                    bulk_g2s(slot + lo, in.p + in.entry(first + lo), (unsigned)(hi - lo) * 16u, &s_full[q]);
                } else {
                    mbar_arrive1(&s_full[q]);
                }
            }
        } else if (tid == 1 && a > 0) {
            slot[0] = in.load(first);
        } else if (tid == 2 && b < n) {
            slot[b] = in.load(first + b);
        }
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
            if (sizeof(T) == 2) mine.zx = to_float((bf16_t)*reinterpret_cast<const volatile unsigned short*>(z + x));
            else mine.zx = to_float(*reinterpret_cast<const volatile float*>(z + x));
        }
    }
    const int xe = token_ok ? x + in.mis : -1;
    const int xl = token_ok ? xe / E - first : -1;      // x's word in the slice (or outside it)
    const uint32_t xbit = token_ok ? 1u << (xe % E) : 0u;
    __syncthreads();

    float m = -INFINITY, s = 0.0f;
    auto batch = [&](int l0, int end) {
        uint4 w[kPolBatch];
        const uint32_t ninf = NegInf<T>::word;
        float bm = -INFINITY;
#pragma unroll
        for (int q = 0; q < kPolBatch; ++q) {
            const int l = l0 + q * kPolThreads + tid;
            if (l < end) w[q] = MODE == 1 ? slot[l] : in.load(first + l);
            else w[q] = make_uint4(ninf, ninf, ninf, ninf);
            if (l == xl) w[q] = word_without<T>(w[q], xbit);
        }
#pragma unroll
        for (int q = 0; q < kPolBatch; ++q) bm = f_max_nan(bm, u4_max_nan<sizeof(T)>(w[q]));
        bm = f_max_nan(bm, m);
        if (bm != m) {
            s = m == -INFINITY ? 0.0f : s * ex2(pol_step(m, bm, c));
            m = bm;
        }
        s += words_sum<T, kPolBatch>(w, m, c);
    };
    bool late = false;
    if (MODE == 1) {
        for (int q = 0; q < kPolChunks; ++q) {
            late |= !mbar_wait(&s_full[q], 0, p.status, kWaitLimitNs);
            const int end = min(n, (q + 1) * per);
            for (int l0 = q * per; l0 < end && !late; l0 += kPolThreads * kPolBatch) batch(l0, end);
        }
        if (late) s_late = 1;
    } else {
        for (int l0 = 0; l0 < n; l0 += kPolThreads * kPolBatch) batch(l0, n);
    }
    if (late) m = NAN;
    {
        float2 v = make_float2(m, s * ref_fix(m, c));
        const float wm = warp_max_nan(v.x);
        v = make_float2(wm, warp_sum(pol_weight(v, wm, c)));
        if (lane == 0) s_warp[warp] = v;
    }
    __syncthreads();
    cluster_wait();
    if (warp == 0) {
        float2 v = lane < kPolWarps ? s_warp[lane] : make_float2(-INFINITY, 0.0f);
        const float wm = warp_max_nan(v.x);
        v = make_float2(wm, warp_sum(pol_weight(v, wm, c)));
        if (lane < (int)size) cluster_put(&s_pair[rank], lane, v);
    }
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
        float2 v = lane < (int)size ? s_pair[lane] : make_float2(-INFINITY, 0.0f);
        const float wm = warp_max_nan(v.x);
        v = make_float2(wm, warp_sum(pol_weight(v, wm, c)));
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
    if (!MODE) return;
    __syncthreads();
    if (MODE == 1 && s_late) {   // what has not arrived may still: out of its way, bounded
        for (int q = 0; q < kPolChunks; ++q) mbar_wait(&s_full[q], 0, p.status, kWaitLimitNs);
    }
    const PolRow r = s_row;
    const float f = -r.factor;
    const bool near = ref_near(r.ref);
    const f2x cc = f2_pack(c, c), mm = f2_pack(-r.ref, -r.ref), ff = f2_pack(f, f);
#pragma unroll 4
    for (int l = tid; l < n; l += kPolThreads) {
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
}

// The cluster's size: slices of 64 KB at most, so that three CTAs share an SM (one loads while
// another forms its gradient), and more CTAs per row where the rows are too few to fill the
// device, down to a batch of words per thread.
template <typename T>
static cudaError_t policy_typed(PolicyParams p, cudaStream_t stream) {
    constexpr int E = 16 / (int)sizeof(T);
    const int words = (p.V + 2 * E - 2) / E;   // whatever the row's offset
    int size = 1;
    while (size < kPolMaxCluster && (words + size - 1) / size > 4096) size *= 2;
    while (size < 8 && (long)p.rows * size < device_sm_count() && words / (2 * size) >= kPolThreads) size *= 2;
    p.slice = (words + size - 1) / size;
    const size_t bytes = (size_t)p.slice * 16;
    const int mode = !p.grad_out ? 0 : (bytes <= 220 * 1024 ? 1 : 2);
    const void* kern = mode == 0 ? (const void*)policy_kernel<T, 0>
                                 : (mode == 1 ? (const void*)policy_kernel<T, 1> : (const void*)policy_kernel<T, 2>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && mode == 1) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows * (unsigned)size);
    cfg.blockDim = dim3(kPolThreads);
    cfg.dynamicSmemBytes = mode == 1 ? bytes : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    e = cudaLaunchKernelExC(&cfg, kern, args);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t policy_launch(PolicyParams p, cudaStream_t stream) {
    return p.dtype == SPEC_BF16 ? policy_typed<bf16_t>(p, stream) : policy_typed<float>(p, stream);
}

}  // namespace spec
