// top_logits.cu - each row's K largest logits and the log-sum-exp of the rest
// (spec_top_logits): a teacher row in the compact form that spec_distill reads.
//
// Two kernels.  top_scan_kernel streams the rows once: a warp-wide load (32 words of 16
// bytes, 512 bytes) is a block, and each block leaves its maximum m and
// s = sum 2^((x - m) log2e / t); the maximum is kept as it is and taken from x before the
// scaling, so that rows filled with the type's lowest value neither overflow nor vanish.  top_pick_kernel, one CTA per row, works on the blocks:
// at most K blocks can hold one of the K largest entries, namely those with the largest
// maxima (equal maxima: the lower block first, since a lower block holds lower indices,
// and ties go to the lowest index).  The same argument on the 16-byte words of those
// blocks leaves at most K words, whose entries are ranked.  Nothing in it depends on how
// the values are distributed: a constant row costs what any row costs.
//
// The rest's sum is made of the blocks that were not chosen and the entries of the chosen
// ones that were not taken; it is never a difference of two sums, so a rest of 1e-12 of
// the row keeps its relative accuracy.
#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kTopThreads = 256;
constexpr int kTopWarps = kTopThreads / 32;
constexpr int kTopBlocksPerWarp = 8;                              // blocks a warp loads at once
constexpr int kTopPiece = kTopWarps * kTopBlocksPerWarp;          // blocks of a CTA

// Blocks of a row of V entries, whatever its offset in its first word.
__host__ __device__ inline int top_blocks(int V, int elt_bytes) {
    const int E = 16 / elt_bytes;
    return ((V + 2 * E - 2) / E + 31) / 32;
}

__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = f_max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <typename T>
__global__ void __launch_bounds__(kTopThreads) top_scan_kernel(TopLogitsParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    const int row = blockIdx.x / p.pieces, piece = blockIdx.x - row * p.pieces;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const RowWords<T> in(reinterpret_cast<const T*>(p.logits) + (long)row * p.ld, p.V);
    const int blk0 = piece * kTopPiece + warp * kTopBlocksPerWarp;
    const uint32_t ninf = NegInf<T>::word;
    uint4 w[kTopBlocksPerWarp];
#pragma unroll
    for (int q = 0; q < kTopBlocksPerWarp; ++q) {
        const int i = (blk0 + q) * 32 + lane;
        w[q] = i < in.n ? in.load(i) : make_uint4(ninf, ninf, ninf, ninf);
    }
#pragma unroll
    for (int q = 0; q < kTopBlocksPerWarp; ++q) {
        const float m = warp_max_nan(u4_max_nan<sizeof(T)>(w[q]));
        float s = 0.0f;
        if (m > -INFINITY) {
#pragma unroll
            for (int k = 0; k < E; ++k) s += ex2((word_entry<T>(w[q], k) - m) * p.scale);
        }
        s = warp_sum(s);
        if (lane == 0 && blk0 + q < p.n_blocks) p.blocks[(long)row * p.n_blocks + blk0 + q] = make_float2(m, s);
    }
}

// Sum of one int per thread over the CTA; `slot` alternates between calls.
__device__ __forceinline__ int cta_sum(int v, int* s_part, int& slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = __reduce_add_sync(0xffffffffu, v);
    int* s = s_part + slot * kTopWarps;
    slot ^= 1;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    int t = 0;
#pragma unroll
    for (int i = 0; i < kTopWarps; ++i) t += s[i];
    return t;
}
// Exclusive prefix over the threads of the CTA.
__device__ __forceinline__ int cta_prefix(int v, int* s_part, int& slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    int* s = s_part + slot * kTopWarps;
    slot ^= 1;
    if (lane == 31) s[warp] = x;
    __syncthreads();
    int base = 0;
    for (int i = 0; i < warp; ++i) base += s[i];
    return base + x - v;
}

// The (at most) K largest of keys[0..n) that are not 0, equal keys by the lower index, as
// ascending indices in list[].  Returns their number; `floor_key` is the smallest of them.
__device__ __forceinline__ int pick_largest(const uint32_t* keys, int n, int K, int* list, uint32_t& floor_key,
                                            int* s_part, int& slot) {
    const int per = (n + kTopThreads - 1) / kTopThreads;
    const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
    uint32_t t = 0;
    for (int bit = 31; bit >= 0; --bit) {   // the largest t with at least K keys >= t
        const uint32_t c = t | (1u << bit);
        int cnt = 0;
        for (int i = lo; i < hi; ++i) cnt += keys[i] >= c ? 1 : 0;
        if (cta_sum(cnt, s_part, slot) >= K) t = c;
    }
    int gt = 0, tie = 0;
    for (int i = lo; i < hi; ++i) {
        gt += keys[i] > t ? 1 : 0;
        tie += (t != 0u && keys[i] == t) ? 1 : 0;
    }
    const int n_gt = cta_sum(gt, s_part, slot), n_tie = cta_sum(tie, s_part, slot);
    const int admit = min(n_tie, K - n_gt);
    int g = cta_prefix(gt, s_part, slot), e = cta_prefix(tie, s_part, slot);
    for (int i = lo; i < hi; ++i) {
        if (keys[i] > t) { list[g + min(e, admit)] = i; ++g; }
        else if (t != 0u && keys[i] == t) {
            if (e < admit) list[g + e] = i;
            ++e;
        }
    }
    floor_key = t;
    __syncthreads();
    return n_gt + admit;
}

// A key that is 0 for -inf and grows with the value otherwise.
__device__ __forceinline__ uint32_t value_key(float x) { return x > -INFINITY ? float_order(x) : 0u; }

// Running maximum m and s = sum w 2^((x - m) c).
struct Run {
    float m = -INFINITY, s = 0.0f;
    __device__ __forceinline__ void add(float x, float w, float c) {
        if (x == -INFINITY) return;
        if (x <= m) { s += w * ex2((x - m) * c); return; }
        s = s * ex2((m - x) * c) + w;
        m = x;
    }
};
// The CTA's total, in every thread.
__device__ __forceinline__ Run run_cta(Run r, float c, float2* s_run) {
    const float M = warp_max(r.m);
    const float s = warp_sum(r.m == -INFINITY ? 0.0f : r.s * ex2((r.m - M) * c));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_run[threadIdx.x >> 5] = make_float2(M, s);
    __syncthreads();
    Run t;
    for (int i = 0; i < kTopWarps; ++i) t.add(s_run[i].x, s_run[i].y, c);
    return t;
}
// ln of the sum
__device__ __forceinline__ float run_log(const Run& r, float inv_t) {
    return r.s > 0.0f ? fmaf(r.m, inv_t, logf(r.s)) : -INFINITY;
}

template <typename T>
__global__ void __launch_bounds__(kTopThreads) top_pick_kernel(TopLogitsParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int KM = SPEC_MAX_TEACHER;
    extern __shared__ __align__(16) uint8_t s_top[];
    uint4* s_words = reinterpret_cast<uint4*>(s_top);                                   // [K][32]
    unsigned long long* s_cand = reinterpret_cast<unsigned long long*>(s_words + p.K * 32);   // [K * 8]
    uint32_t* s_keys = reinterpret_cast<uint32_t*>(s_cand + p.K * 8);                    // [max(n_blocks, K * 32)]
    __shared__ int s_blk[KM], s_word[KM], s_part[2 * kTopWarps], s_n, s_bad;
    __shared__ unsigned long long s_kth;
    __shared__ float2 s_run[kTopWarps];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.K;
    const RowWords<T> in(reinterpret_cast<const T*>(p.logits) + (long)row * p.ld, p.V);
    const float2* blk = p.blocks + (long)row * p.n_blocks;
    float* values = p.values_out + (long)row * K;
    int32_t* ids = p.ids_out + (long)row * K;
    int slot = 0;

    if (tid == 0) { s_n = 0; s_bad = 0; s_kth = 0ull; }
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < p.n_blocks; i += kTopThreads) {
        const float m = blk[i].x;
        bad |= bad_logit(m);
        s_keys[i] = value_key(m);
    }
    if (bad) s_bad = 1;
    __syncthreads();
    if (s_bad) {
        for (int k = tid; k < K; k += kTopThreads) { values[k] = NAN; ids[k] = -1; }
        if (tid == 0) {
            p.tail_out[row] = NAN;
            if (p.lse_out) p.lse_out[row] = NAN;
            atomicOr(p.status, SPEC_DEV_NONFINITE);
        }
        return;
    }
    uint32_t floor_key;
    const int nb = pick_largest(s_keys, p.n_blocks, K, s_blk, floor_key, s_part, slot);
    // the sum of the blocks that were not chosen
    Run rest;
    for (int i = tid; i < p.n_blocks; i += kTopThreads) {
        int lo = 0, hi = nb;   // is i in the ascending list?
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_blk[mid] < i) lo = mid + 1;
            else hi = mid;
        }
        if (lo < nb && s_blk[lo] == i) continue;
        const float2 ms = blk[i];
        rest.add(ms.x, ms.y, p.scale);
    }
    __syncthreads();
    const uint32_t ninf = NegInf<T>::word;
    for (int q = warp; q < nb; q += kTopWarps) {
        const int i = s_blk[q] * 32 + lane;
        const uint4 w = i < in.n ? in.load(i) : make_uint4(ninf, ninf, ninf, ninf);
        s_words[q * 32 + lane] = w;
        s_keys[q * 32 + lane] = value_key(u4_max_nan<sizeof(T)>(w));
    }
    __syncthreads();
    const int nw = pick_largest(s_keys, nb * 32, K, s_word, floor_key, s_part, slot);
    for (int i = tid; i < nw * E; i += kTopThreads) {
        const int q = s_word[i / E], k = i % E;
        const float x = word_entry<T>(s_words[q], k);
        const uint32_t vk = value_key(x);
        if (vk != 0u && vk >= floor_key) {
            const int e = in.entry(s_blk[q >> 5] * 32 + (q & 31)) + k;
            s_cand[atomicAdd(&s_n, 1)] = argmax_key(x, (uint32_t)e);
        }
    }
    __syncthreads();
    const int n = s_n;
    for (int i = tid; i < n; i += kTopThreads) {
        const unsigned long long key = s_cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += s_cand[j] > key ? 1 : 0;
        if (rank < K) {
            values[rank] = key_value(key);
            ids[rank] = (int)key_index(key);
            if (rank == K - 1) s_kth = key;
        }
    }
    for (int k = n + tid; k < K; k += kTopThreads) { values[k] = -INFINITY; ids[k] = -1; }
    __syncthreads();
    const unsigned long long kth = s_kth;   // 0 when every finite entry was taken
    Run taken;
    for (int i = tid; i < nb * 32; i += kTopThreads) {
        const int e = in.entry(s_blk[i >> 5] * 32 + (i & 31));
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const float x = word_entry<T>(s_words[i], k);
            if (argmax_key(x, (uint32_t)(e + k)) >= kth) taken.add(x, 1.0f, p.scale);
            else rest.add(x, 1.0f, p.scale);
        }
    }
    const Run r = run_cta(rest, p.scale, s_run);
    Run a = run_cta(taken, p.scale, s_run);
    if (tid == 0) {
        p.tail_out[row] = run_log(r, p.inv_t);
        a.add(r.m, r.s, p.scale);
        if (p.lse_out) p.lse_out[row] = run_log(a, p.inv_t);
        if (!(a.s > 0.0f)) atomicOr(p.status, SPEC_DEV_NONFINITE);   // no finite entry
    }
}

size_t top_logits_workspace_bytes(int rows, int V) {
    return kWsHeaderBytes + (size_t)rows * top_blocks(V, 4) * sizeof(float2);
}

template <typename T>
static cudaError_t top_launch(TopLogitsParams p, cudaStream_t stream) {
    p.n_blocks = top_blocks(p.V, sizeof(T));
    p.pieces = (p.n_blocks + kTopPiece - 1) / kTopPiece;
    const long grid = (long)p.rows * p.pieces;
    if (grid > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    top_scan_kernel<T><<<(unsigned)grid, kTopThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int nkeys = p.n_blocks > p.K * 32 ? p.n_blocks : p.K * 32;
    const size_t smem = (size_t)p.K * 32 * 16 + (size_t)p.K * 8 * 8 + (size_t)nkeys * 4;
    const cudaError_t a = cudaFuncSetAttribute(top_pick_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (a != cudaSuccess) return a;
    top_pick_kernel<T><<<p.rows, kTopThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t top_logits_launch(TopLogitsParams p, void* ws, cudaStream_t stream) {
    p.status = &reinterpret_cast<WsHeader*>(ws)->status;
    p.blocks = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(ws) + kWsHeaderBytes);
    return p.dtype == SPEC_BF16 ? top_launch<bf16_t>(p, stream) : top_launch<float>(p, stream);
}

}  // namespace spec
