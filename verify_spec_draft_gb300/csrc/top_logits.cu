// top_logits.cu - each row's K largest logits and the log-sum-exp of the rest
// (spec_top_logits): a teacher row in the compact form that spec_distill reads.
//
// CTAs stream pieces of the rows: a warp-wide load (32 words of 16 bytes) is a block, or eight of
// them where a row has fewer than twice K, and each block leaves its maximum and the sum of
// its weights relative to it (row_words.cuh).  Then each row is picked from: the K largest
// entries lie in blocks whose maxima are among the K largest, so a bisection over the block
// maxima that ends as soon as K to K + 32 of them lie at or above the pivot names the blocks
// to look at again, and their entries at or above the pivot (a few more than K as a rule)
// are ranked.
// Equal values need care: a row can hold thousands of entries at the pivot.  Where more
// blocks or entries than there is room for lie at or above it, the choice is made exact:
// the blocks (then the 16-byte words of those blocks) with the K largest maxima, equal ones by
// the lower index, since a lower block holds lower indices and ties go to the lowest index.
// That leaves at most K words, whatever the values.
//
// The rest's sum is made of the blocks that were not chosen and the entries of the chosen
// ones that were not taken; it is never a difference of two sums, so a rest of 1e-12 of
// the row keeps its relative accuracy.
//
// Bound: 256 rows of 248,320 bf16, K 64, take 30.4 us, 4.2 TB/s of what has to be read and 62 %
// of a copy's rate.  The scan goes at the memory's pace (24 us by itself, from cold caches,
// 5.3 TB/s); the picks are latency, some 8 us of steps that wait for one another (the maxima,
// the bisection, the chosen blocks, the ranks) with a fifth of the warps there.  A full
// selection over the block maxima took 76 us in all, reading the chosen blocks twice 61.
#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kTopThreads = 256;
constexpr int kTopWarps = kTopThreads / 32;
constexpr int kTopBatch = 8;                       // blocks a warp loads at once
constexpr int kTopSlack = 32;                      // blocks beyond K that the bisection may leave
constexpr int kTopBlkMax = SPEC_MAX_TEACHER + kTopSlack;
// Rows from which the picks are a launch of their own, not the last piece's CTA's: of 248,320
// bf16, K 20, 256 rows took 31.0 us that way instead of 36.9, 64 rows 15.0 instead of 16.8; 1 and
// 16 rows 10.9 and 11.6 instead of 11.4 and 12.6, but a second launch costs the host 1.5 us, and
// the host is what holds so short a call.
constexpr int kTopApart = 32;
// Blocks per entry asked for, at least (smaller blocks otherwise): 256 rows of 32,000, K 128,
// took 17 us where 125 blocks of 32 words took 103; 64 rows of 151,936, K 128, with their 594
// blocks took 18 us where blocks of 4 words took 23.
constexpr int kTopMany = 2;
constexpr int kTopAgain = 4;                       // words a thread holds when it looks again
constexpr int kTopRecords = 4;                     // blocks' records a thread loads at once
constexpr int kTopCandMax = SPEC_MAX_TEACHER * 8;  // entries to rank

// Blocks of `lanes` words of a row of V entries, whatever its offset in its first word, in
// whole warps' loads.
__host__ __device__ inline int top_blocks(int V, int elt_bytes, int lanes) {
    const int E = 16 / elt_bytes;
    return ((V + 2 * E - 2) / E + 31) / 32 * (32 / lanes);
}

// The sums over the warp of eight values per lane, two lanes' halves at a time: lane l ends
// with the sum of value (l >> 2).
__device__ __forceinline__ float warp_sum8(float (&v)[8]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 4, o = 16; h >= 1; h >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float send = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
    return v[0];
}

// s_keys: the blocks' keys [n_blocks] and sums [n_blocks], then room for 32 words per entry.
template <typename T, bool ALIGNED, int LANES>
__device__ __forceinline__ void top_pick(const TopLogitsParams& p, int row, uint32_t* s_keys);

// The blocks of one piece, then, in the CTA that finishes its row's last piece, the pick.
template <typename T, bool ALIGNED, int LANES>
__global__ void __launch_bounds__(kTopThreads) top_kernel(TopLogitsParams p) {
    static_assert(LANES == 32 || LANES == 4, "a block is a warp's load or an eighth of it");
    extern __shared__ __align__(16) uint32_t s_keys[];
    const int row = blockIdx.x / p.pieces, piece = blockIdx.x - row * p.pieces;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SegWords<T, ALIGNED> in(reinterpret_cast<const T*>(p.logits) + (long)row * p.ld, p.V);
    const int blk0 = (piece * kTopWarps + warp) * p.batch;   // batch <= kTopBatch loads of this warp
    const int n = in.n();
    const uint32_t ninf = NegInf<T>::word;
    uint4 w[kTopBatch];
    if (p.batch == kTopBatch && (blk0 + kTopBatch) * 32 <= n) {
#pragma unroll
        for (int q = 0; q < kTopBatch; ++q) w[q] = in.load((blk0 + q) * 32 + lane);
    } else {
#pragma unroll
        for (int q = 0; q < kTopBatch; ++q) {
            const int i = (blk0 + q) * 32 + lane;
            w[q] = q < p.batch && i < n ? in.load(i) : make_uint4(ninf, ninf, ninf, ninf);
        }
    }
    float m[kTopBatch], s[kTopBatch];
#pragma unroll
    for (int q = 0; q < kTopBatch; ++q) {
        m[q] = u4_max_nan<sizeof(T)>(w[q]);
        if (LANES == 32) {
            m[q] = warp_max_nan(m[q]);
        } else {
            m[q] = f_max_nan(m[q], __shfl_xor_sync(0xffffffffu, m[q], 1));
            m[q] = f_max_nan(m[q], __shfl_xor_sync(0xffffffffu, m[q], 2));
        }
        const uint4 one[1] = {w[q]};
        s[q] = words_sum<T, 1>(one, m[q], p.scale);
    }
    float2* out = p.blocks + (long)row * p.n_blocks;
    if (LANES == 32) {
        const float sum = warp_sum8(s);
        const int mine = lane >> 2;
        float mx = m[0];
#pragma unroll
        for (int q = 1; q < kTopBatch; ++q) mx = mine == q ? m[q] : mx;
        if ((lane & 3) == 0 && mine < p.batch && blk0 + mine < p.n_blocks) __stcg(&out[blk0 + mine], make_float2(mx, sum * ref_fix(mx, p.scale)));
    } else {
#pragma unroll
        for (int q = 0; q < kTopBatch; ++q) {
            s[q] += __shfl_xor_sync(0xffffffffu, s[q], 1);
            s[q] += __shfl_xor_sync(0xffffffffu, s[q], 2);
            const int b = (blk0 + q) * 8 + (lane >> 2);
            if ((lane & 3) == 0 && q < p.batch && b < p.n_blocks) __stcg(&out[b], make_float2(m[q], s[q] * ref_fix(m[q], p.scale)));
        }
    }
    if (p.pick_apart) {
        pdl_launch_dependents();
        return;
    }
    if (!last_block_done(&p.done[row], (unsigned)p.pieces)) return;
    if (threadIdx.x == 0) p.done[row] = 0u;
    top_pick<T, ALIGNED, LANES>(p, row, s_keys);
}

// The picks of all rows, launched behind the scan as its programmatic dependent.
// Rows that a SM picks from at once.  Four leave the registers to request words ahead (256 rows of
// 248,320 bf16: 30.8 us, with five 31.9), which rows that are not whole words have no use for (611
// rows of 50,257 float32: 42 us with four, 38 with five).
template <typename T, bool ALIGNED, int LANES>
__global__ void __launch_bounds__(kTopThreads, ALIGNED ? 4 : 5) top_pick_kernel(TopLogitsParams p) {
    extern __shared__ __align__(16) uint32_t s_keys[];
    pdl_wait_primary();
    top_pick<T, ALIGNED, LANES>(p, blockIdx.x, s_keys);
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
// Two such sums.
__device__ __forceinline__ int2 cta_sums(int a, int b, int2* s_pair, int& slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = __reduce_add_sync(0xffffffffu, a);
    b = __reduce_add_sync(0xffffffffu, b);
    int2* s = s_pair + slot * kTopWarps;
    slot ^= 1;
    if (lane == 0) s[warp] = make_int2(a, b);
    __syncthreads();
    int2 t = make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < kTopWarps; ++i) {
        const int2 v = s[i];
        t.x += v.x;
        t.y += v.y;
    }
    return t;
}
// Exclusive prefix over the threads of the CTA, and the total.
__device__ __forceinline__ int cta_prefix(int v, int& total, int* s_part, int& slot) {
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
    int base = 0, t = 0;
#pragma unroll
    for (int i = 0; i < kTopWarps; ++i) {
        if (i == warp) base = t;
        t += s[i];
    }
    total = t;
    return base + x - v;
}

// The (at most) K largest of keys[0..n) that are not 0, equal keys by the lower index, as
// ascending indices in list[].  Returns their number; `floor_key` is the smallest of them.
__device__ __noinline__ int pick_largest(const uint32_t* keys, int n, int K, int* list, uint32_t& floor_key,
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
    int n_gt, n_tie;
    int g = cta_prefix(gt, n_gt, s_part, slot), e = cta_prefix(tie, n_tie, s_part, slot);
    const int admit = min(n_tie, K - n_gt);
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

// Words of a block: 32, or 4 where that leaves a row fewer than kTopMany K blocks.
__host__ __device__ inline int top_lanes(int V, int elt_bytes, int K) {
    return top_blocks(V, elt_bytes, 32) < kTopMany * K ? 4 : 32;
}

// A key that is 0 for -inf and grows with the value otherwise.
__device__ __forceinline__ uint32_t value_key(float x) { return x > -INFINITY ? float_order(x) : 0u; }

// The least value with at least this key.
__device__ __forceinline__ float key_floor(uint32_t key) {
    return key < float_order(-3.402823466e38f) ? -3.402823466e38f : order_float(key);
}

// Running maximum m and the sum of weights relative to it.
struct Run {
    float m = -INFINITY, s = 0.0f;
    __device__ __forceinline__ void raise(float x, float c) {
        if (!(x > m)) return;
        s = m == -INFINITY ? 0.0f : s * ex2(ref_rel(m, x, c));
        m = x;
    }
    __device__ __forceinline__ void entry(float x, float c) {   // one entry
        if (x == -INFINITY) return;
        raise(x, c);
        s += ex2(ref_rel(x, m, c));
    }
    __device__ __forceinline__ void sum(float x, float w, float c) {   // a sum relative to x
        if (x == -INFINITY) return;
        raise(x, c);
        s += w * ex2(ref_rel(x, m, c));
    }
    template <typename T, int N>
    __device__ __forceinline__ void words(const uint4 (&w)[N], float mx, float c) {   // their maximum is mx
        raise(mx, c);
        s += words_sum<T, N>(w, m, c) * ref_fix(m, c);
    }
};
// The CTA's totals of two runs, in the first warp.
__device__ __forceinline__ void runs_cta(Run& x, Run& y, float c, float4* s_run) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float mx = warp_max(x.m), my = warp_max(y.m);
    const float sx = warp_sum(x.m == -INFINITY ? 0.0f : x.s * ex2(ref_rel(x.m, mx, c)));
    const float sy = warp_sum(y.m == -INFINITY ? 0.0f : y.s * ex2(ref_rel(y.m, my, c)));
    if (lane == 0) s_run[warp] = make_float4(mx, sx, my, sy);
    __syncthreads();
    if (warp != 0) return;
    const float4 v = lane < kTopWarps ? s_run[lane] : make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
    x.m = warp_max(v.x);
    y.m = warp_max(v.z);
    x.s = warp_sum(v.x == -INFINITY ? 0.0f : v.y * ex2(ref_rel(v.x, x.m, c)));
    y.s = warp_sum(v.z == -INFINITY ? 0.0f : v.w * ex2(ref_rel(v.z, y.m, c)));
}
// ln of the sum
__device__ __forceinline__ float run_log(const Run& r, float inv_t) {
    return r.s > 0.0f ? ref_log(r.m, r.s, inv_t) : -INFINITY;
}

// The indices of keys[0..n) at or above `t` in list[], in an order that depends on them alone.
__device__ __forceinline__ void list_above(const uint32_t* keys, int n, uint32_t t, int* list, int* s_part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int cnt = 0;
    for (int i0 = 0; i0 < n; i0 += kTopThreads) {
        const int i = i0 + threadIdx.x;
        cnt += __popc(__ballot_sync(0xffffffffu, i < n && keys[i] >= t));
    }
    __syncthreads();
    if (lane == 0) s_part[warp] = cnt;
    __syncthreads();
    int at = 0;
    for (int i = 0; i < warp; ++i) at += s_part[i];
    for (int i0 = 0; i0 < n; i0 += kTopThreads) {
        const int i = i0 + threadIdx.x;
        const bool in = i < n && keys[i] >= t;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (in) list[at + __popc(who & ((1u << lane) - 1u))] = i;
        at += __popc(who);
    }
    __syncthreads();
}

template <typename T, bool ALIGNED, int LANES>
__device__ __forceinline__ void top_pick(const TopLogitsParams& p, int row, uint32_t* s_keys) {
    constexpr int E = 16 / (int)sizeof(T), PER = 32 / LANES;   // blocks of a warp's load
    __shared__ unsigned long long s_cand[kTopCandMax];
    __shared__ int s_word[kTopCandMax];                      // listed words to look at, then ranks
    __shared__ unsigned s_hit[kTopBlkMax];
    __shared__ int s_blk[kTopBlkMax], s_part[2 * kTopWarps], s_bad;
    __shared__ int2 s_pair[2 * kTopWarps];
    __shared__ uint32_t s_lo, s_hi;
    __shared__ unsigned long long s_kth;
    __shared__ float4 s_run[kTopWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.K;
    const SegWords<T, ALIGNED> in(reinterpret_cast<const T*>(p.logits) + (long)row * p.ld, p.V);
    const float2* blk = p.blocks + (long)row * p.n_blocks;
    float* values = p.values_out + (long)row * K;
    int32_t* ids = p.ids_out + (long)row * K;
    const uint32_t ninf = NegInf<T>::word;
    auto word_at = [&](int b, int l) {   // word l of block b
        const int i = b * LANES + l;
        return i < in.n() ? in.load(i) : make_uint4(ninf, ninf, ninf, ninf);
    };
    float* s_sums = reinterpret_cast<float*>(s_keys + p.n_blocks);
    int slot = 0;

    if (tid == 0) {
        s_bad = 0;
        s_kth = 0ull;
        s_lo = 0xffffffffu;
        s_hi = 0u;
    }
    __syncthreads();
    bool bad = false;
    uint32_t klo = 0xffffffffu, khi = 0u;
    int cnt = 0;
    for (int i0 = tid; i0 < p.n_blocks; i0 += kTopRecords * kTopThreads) {
        float2 ms[kTopRecords];
#pragma unroll
        for (int h = 0; h < kTopRecords; ++h) {
            const int i = i0 + h * kTopThreads;
            ms[h] = i < p.n_blocks ? __ldcg(&blk[i]) : make_float2(-INFINITY, 0.0f);
        }
#pragma unroll
        for (int h = 0; h < kTopRecords; ++h) {
            const int i = i0 + h * kTopThreads;
            bad |= bad_logit(ms[h].x);
            const uint32_t key = value_key(ms[h].x);
            if (i < p.n_blocks) {
                s_keys[i] = key;
                s_sums[i] = ms[h].y;
            }
            if (key) {
                klo = min(klo, key);
                khi = max(khi, key);
                ++cnt;
            }
        }
    }
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
    if (lane == 0) {
        atomicMin(&s_lo, klo);
        atomicMax(&s_hi, khi);
    }
    if (bad) s_bad = 1;
    int n_above = cta_sum(cnt, s_part, slot);   // blocks with a finite entry
    if (s_bad) {
        for (int k = tid; k < K; k += kTopThreads) { values[k] = NAN; ids[k] = -1; }
        if (tid == 0) {
            p.tail_out[row] = NAN;
            if (p.lse_out) p.lse_out[row] = NAN;
            atomicOr(p.status, SPEC_DEV_NONFINITE);
        }
        return;
    }
    // a pivot with K to K + kTopSlack blocks at or above it: count(lo) = n_above >= K > count(hi),
    // the range cut to a quarter at a time
    uint32_t lo = n_above ? s_lo : 1u, hi = n_above ? s_hi + 1u : 1u;
    while (n_above > K + kTopSlack && hi - lo > 1u) {
        const uint32_t d = (hi - lo) / 4u;
        const uint32_t t1 = d ? lo + d : lo + 1u, t2 = d ? t1 + d : t1, t3 = d ? t2 + d : t1;
        int c12 = 0, c3 = 0;
        for (int i = tid; i < p.n_blocks; i += kTopThreads) {
            const uint32_t key = s_keys[i];
            c12 += (key >= t1 ? 1 : 0) + (key >= t2 ? 65536 : 0);
            c3 += key >= t3 ? 1 : 0;
        }
        const int2 c = cta_sums(c12, c3, s_pair, slot);
        const int c1 = c.x & 0xffff, c2 = c.x >> 16;
        c3 = c.y;
        if (c3 >= K) { lo = t3; n_above = c3; }
        else if (c2 >= K) { lo = t2; n_above = c2; hi = t3; }
        else if (c1 >= K) { lo = t1; n_above = c1; hi = t2; }
        else hi = t1;
    }
    __syncthreads();
    int nb = n_above;
    const bool exact_blocks = n_above > K + kTopSlack;
    uint32_t floor_key = nb >= K ? lo : 1u;   // fewer than K blocks bound nothing: every finite entry
    if (!exact_blocks) list_above(s_keys, p.n_blocks, lo, s_blk, s_part);
    else nb = pick_largest(s_keys, p.n_blocks, K, s_blk, floor_key, s_part, slot);

    // the chosen blocks once more: entries at or above the pivot are candidates, the others
    // belong to the rest
    Run rest, taken;
    // The chosen blocks' words in the list's order, 32 at a time (a warp's load): `u`, lane.
    auto listed_word = [&](int u, int l) {
        const int i = u * PER + l / LANES;
        return i < nb ? word_at(s_blk[i], l % LANES) : make_uint4(ninf, ninf, ninf, ninf);
    };
    auto load_blocks = [&](int u0, uint4 (&w)[kTopAgain]) {
#pragma unroll
        for (int h = 0; h < kTopAgain; ++h) w[h] = listed_word(u0 + h * kTopWarps, lane);
    };
    auto over_blocks = [&](auto&& body) {   // a warp's share of them, kTopAgain loads at a time
        for (int u0 = warp; u0 * PER < nb; u0 += kTopAgain * kTopWarps) {
            uint4 w[kTopAgain];
            load_blocks(u0, w);
            body(u0, w);
        }
    };
    // Entries of listed words from `least` on become candidates, in the words' order; `body` gets
    // the word without them.  Returns the candidates' number (which may pass the room).
    auto candidates = [&](int n_words, float least, auto&& body) {
        int n = 0;
        for (int i0 = 0; i0 < n_words; i0 += kTopThreads) {
            const int i = i0 + tid, at_word = i < n_words ? s_word[i] : 0;
            uint4 w = make_uint4(ninf, ninf, ninf, ninf);
            if (i < n_words) w = listed_word(at_word >> 5, at_word & 31);
            uint32_t above = 0u;
#pragma unroll
            for (int k = 0; k < E; ++k) above |= word_entry<T>(w, k) >= least ? 1u << k : 0u;
            int more;
            int at = n + cta_prefix(__popc(above), more, s_part, slot);
            n += more;
            const int e0 = in.entry(s_blk[(at_word >> 5) * PER + (at_word & 31) / LANES] * LANES + (at_word & 31) % LANES);
            for (uint32_t a = above; a; a &= a - 1u, ++at) {
                const int k = __ffs(a) - 1;
                if (at < kTopCandMax) s_cand[at] = argmax_key(word_pick<T>(w, k), (uint32_t)(e0 + k));
            }
            body(word_without<T>(w, above));
        }
        __syncthreads();
        return n;
    };
    // the words that hold an entry at or above the pivot are noted, the others summed
    float least = key_floor(floor_key);   // (a key of 1 stands for the lowest float: every finite entry)
    // The words behind are requested before these are worked on where the loads are plain ones;
    // the others' registers would take places from other rows (see top_pick_kernel).
    constexpr bool AHEAD = ALIGNED;
    uint4 w[kTopAgain], ahead[kTopAgain];
    load_blocks(warp, w);
    // meanwhile the sums of the blocks that are not looked at again
    Run others;
    if (!exact_blocks) {
        uint32_t most = 0u;
        for (int i = tid; i < p.n_blocks; i += kTopThreads) {
            const uint32_t key = s_keys[i];
            if (key < lo) most = max(most, key);
        }
        if (most) {
            others.m = order_float(most);
            for (int i = tid; i < p.n_blocks; i += kTopThreads) {
                const uint32_t key = s_keys[i];
                if (key && key < lo) others.s += s_sums[i] * ex2(ref_rel(order_float(key), others.m, p.scale));
            }
        }
    }
    for (int u0 = warp; u0 * PER < nb; u0 += kTopAgain * kTopWarps) {
        if (AHEAD) load_blocks(u0 + kTopAgain * kTopWarps, ahead);
        float mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < kTopAgain; ++h) {
            const float wm = u4_max_nan<sizeof(T)>(w[h]);
            const bool hit = wm >= least;
            const unsigned who = __ballot_sync(0xffffffffu, hit);
            if (lane == 0 && (u0 + h * kTopWarps) * PER < nb) s_hit[u0 + h * kTopWarps] = who;
            if (hit) w[h] = make_uint4(ninf, ninf, ninf, ninf);
            else mx = fmaxf(mx, wm);
        }
        rest.words<T, kTopAgain>(w, mx, p.scale);
        if (AHEAD) {
#pragma unroll
            for (int h = 0; h < kTopAgain; ++h) w[h] = ahead[h];
        } else {
            load_blocks(u0 + kTopAgain * kTopWarps, w);
        }
    }
    __syncthreads();
    // then looked at in parallel, a thread each
    unsigned who = tid * PER < nb ? s_hit[tid] : 0u;
    int n_hit;
    int at = cta_prefix(__popc(who), n_hit, s_part, slot);
    for (; who; who &= who - 1u, ++at)
        if (at < kTopCandMax) s_word[at] = tid * 32 + __ffs(who) - 1;
    __syncthreads();
    int n = kTopCandMax + 1;
    if (n_hit <= kTopCandMax)
        n = candidates(n_hit, least, [&](const uint4& w) {
            const uint4 one[1] = {w};
            rest.words<T, 1>(one, u4_max_nan<sizeof(T)>(w), p.scale);
        });
    const bool exact_words = n > kTopCandMax;
    if (exact_words) {
        // equal values in numbers: the K largest word maxima of (exactly) K blocks, in the
        // blocks' order
        __syncthreads();
        if (!exact_blocks) nb = pick_largest(s_keys, p.n_blocks, K, s_blk, floor_key, s_part, slot);
        __syncthreads();
        uint32_t* s_wkeys = s_keys + 2 * p.n_blocks;   // [K * LANES]
        over_blocks([&](int u0, uint4 (&w)[kTopAgain]) {
#pragma unroll
            for (int h = 0; h < kTopAgain; ++h) {
                const int i = (u0 + h * kTopWarps) * 32 + lane;
                if (i < nb * LANES) s_wkeys[i] = value_key(u4_max_nan<sizeof(T)>(w[h]));
            }
        });
        __syncthreads();
        const int nw = pick_largest(s_wkeys, nb * LANES, K, s_word, floor_key, s_part, slot);
        n = candidates(nw, key_floor(floor_key), [](const uint4&) {});
    }
    // Many more candidates than K (few blocks, or equal values): a bisection over them first, so
    // that few are ranked.
    uint32_t pivot = 0u;
    if (n > 2 * K + kTopSlack) {
        uint32_t a = 0xffffffffu, b = 0u;
        for (int i = tid; i < n; i += kTopThreads) {
            a = min(a, (uint32_t)(s_cand[i] >> 32));
            b = max(b, (uint32_t)(s_cand[i] >> 32));
        }
        if (tid == 0) {
            s_lo = 0xffffffffu;
            s_hi = 0u;
        }
        __syncthreads();
        atomicMin(&s_lo, a);
        atomicMax(&s_hi, b);
        __syncthreads();
        uint32_t l = s_lo, h = s_hi;   // count(l) >= K; stops where count(h + 1) < K
        int c = n;
        while (l < h && c > K + kTopSlack) {
            const uint32_t mid = l + (h - l) / 2u + 1u;
            int cnt = 0;
            for (int i = tid; i < n; i += kTopThreads) cnt += (uint32_t)(s_cand[i] >> 32) >= mid ? 1 : 0;
            cnt = cta_sum(cnt, s_part, slot);
            if (cnt >= K) { l = mid; c = cnt; }
            else h = mid - 1u;
        }
        pivot = l;
    }
    // ranks: as many threads share a candidate's comparisons, one to eight of them, as leave
    // one pass over the candidates
    const int share = n > kTopThreads / 2 ? 0 : (n > kTopThreads / 4 ? 1 : (n > kTopThreads / 8 ? 2 : 3));
    for (int i0 = 0; i0 < n; i0 += kTopThreads >> share) {
        const int i = i0 + (tid >> share);
        const unsigned long long key = i < n ? s_cand[i] : 0ull;
        const bool ranked = i < n && (uint32_t)(key >> 32) >= pivot;
        int r = 0;
        if (__any_sync(0xffffffffu, ranked)) {
#pragma unroll 8
            for (int j = tid & ((1 << share) - 1); j < n; j += 1 << share) r += s_cand[j] > key ? 1 : 0;
        }
        for (int o = 0; o < share; ++o) r += __shfl_xor_sync(0xffffffffu, r, 1 << o);
        if ((tid & ((1 << share) - 1)) == 0 && i < n) s_word[i] = ranked ? r : K;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kTopThreads) {
        const unsigned long long key = s_cand[i];
        const int rank = s_word[i];
        const float x = key_value(key);
        if (rank < K) {
            values[rank] = x;
            ids[rank] = (int)key_index(key);
            if (rank == K - 1) s_kth = key;
            taken.entry(x, p.scale);
        } else if (!exact_words) {
            rest.entry(x, p.scale);
        }
    }
    __syncthreads();
    for (int k = n + tid; k < K; k += kTopThreads) { values[k] = -INFINITY; ids[k] = -1; }
    if (exact_words) {   // the chosen blocks' entries that were not taken, over again
        const unsigned long long kth = s_kth;   // 0 when every finite entry was taken
        rest = Run();
        over_blocks([&](int u0, uint4 (&w)[kTopAgain]) {
            float mx = -INFINITY;
#pragma unroll
            for (int h = 0; h < kTopAgain; ++h) {
                const int i = (u0 + h * kTopWarps) * PER + lane / LANES;
                if (i >= nb) continue;
                const int e = in.entry(s_blk[i] * LANES + lane % LANES);
                uint32_t taken_bits = 0u;
#pragma unroll
                for (int k = 0; k < E; ++k)
                    taken_bits |= argmax_key(word_entry<T>(w[h], k), (uint32_t)(e + k)) >= kth ? 1u << k : 0u;
                w[h] = word_without<T>(w[h], taken_bits);
                mx = fmaxf(mx, u4_max_nan<sizeof(T)>(w[h]));
            }
            rest.words<T, kTopAgain>(w, mx, p.scale);
        });
    }
    if (exact_blocks || exact_words) {   // the blocks that were not looked at again: not in the ascending list
        if (exact_words) others = Run();
        for (int i = tid; i < p.n_blocks; i += kTopThreads) {
            int a = 0, b = nb;
            while (a < b) {
                const int mid = (a + b) >> 1;
                if (s_blk[mid] < i) a = mid + 1;
                else b = mid;
            }
            if (!(a < nb && s_blk[a] == i) && s_keys[i]) others.sum(order_float(s_keys[i]), s_sums[i], p.scale);
        }
    }
    rest.sum(others.m, others.s, p.scale);
    runs_cta(rest, taken, p.scale, s_run);
    if (tid == 0) {
        p.tail_out[row] = run_log(rest, p.inv_t);
        taken.sum(rest.m, rest.s, p.scale);
        if (p.lse_out) p.lse_out[row] = run_log(taken, p.inv_t);
        if (!(taken.s > 0.0f)) atomicOr(p.status, SPEC_DEV_NONFINITE);   // no finite entry
    }
}

// A row's blocks' keys and sums and, where its ties need them, the chosen blocks' words.
static size_t top_smem(int n_blocks, int K, int lanes) { return ((size_t)n_blocks * 2 + (size_t)K * lanes) * 4; }
constexpr int kTopSmemPlain = 28 * 1024;   // what a kernel gets beside its own arrays without being asked for more
// The most that any call needs, float32 rows of SPEC_MAX_V_TEACHER.  The attribute is always set to
// this: it belongs to the kernel, and another host thread may set it between a call's own setting and
// its launch.
constexpr int kTopSmemMost = 81928;

size_t top_logits_workspace_bytes(int rows, int K, int V) {
    const int f32 = top_lanes(V, 4, K), bf16 = top_lanes(V, 2, K);
    const int a = top_blocks(V, 4, f32), b = top_blocks(V, 2, bf16);
    return kWsHeaderBytes + align256((size_t)rows * sizeof(unsigned)) + (size_t)rows * (a > b ? a : b) * sizeof(float2);
}

template <typename T, int LANES>
static cudaError_t top_launch_lanes(TopLogitsParams p, cudaStream_t stream) {
    p.n_blocks = top_blocks(p.V, sizeof(T), LANES);
    const int loads = p.n_blocks * LANES / 32;
    // a warp's loads: eight (the most in flight) unless that leaves SMs without a CTA
    p.batch = kTopBatch;
    while (p.batch > 1 && (long)p.rows * ((loads + kTopWarps * p.batch - 1) / (kTopWarps * p.batch)) < device_sm_count())
        p.batch /= 2;
    p.pieces = (loads + kTopWarps * p.batch - 1) / (kTopWarps * p.batch);
    const long grid = (long)p.rows * p.pieces;
    if (grid > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    const bool aligned = SegWords<T, true>::fits(p.ld, p.V);
    const void* scan = aligned ? (const void*)top_kernel<T, true, LANES> : (const void*)top_kernel<T, false, LANES>;
    const auto pick = aligned ? top_pick_kernel<T, true, LANES> : top_pick_kernel<T, false, LANES>;
    const size_t smem = top_smem(p.n_blocks, p.K, LANES);
    if (smem > kTopSmemMost) return cudaErrorInvalidConfiguration;
    p.pick_apart = p.rows >= kTopApart;
    if (smem > kTopSmemPlain) {
        const cudaError_t e = cudaFuncSetAttribute(p.pick_apart ? (const void*)pick : scan, cudaFuncAttributeMaxDynamicSharedMemorySize, kTopSmemMost);
        if (e != cudaSuccess) return e;
    }
    void* args[] = {&p};
    const cudaError_t e = cudaLaunchKernel(scan, dim3((unsigned)grid), dim3(kTopThreads), args, p.pick_apart ? 0 : smem, stream);
    if (e != cudaSuccess || !p.pick_apart) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows);
    cfg.blockDim = dim3(kTopThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pick, p);
}
template <typename T>
static cudaError_t top_launch(const TopLogitsParams& p, cudaStream_t stream) {
    return top_lanes(p.V, sizeof(T), p.K) == 32 ? top_launch_lanes<T, 32>(p, stream) : top_launch_lanes<T, 4>(p, stream);
}

cudaError_t top_logits_launch(TopLogitsParams p, void* ws, cudaStream_t stream) {
    p.status = &reinterpret_cast<WsHeader*>(ws)->status;
    uint8_t* b = reinterpret_cast<uint8_t*>(ws) + kWsHeaderBytes;
    p.done = reinterpret_cast<unsigned*>(b);
    p.blocks = reinterpret_cast<float2*>(b + align256((size_t)p.rows * sizeof(unsigned)));
    return p.dtype == SPEC_BF16 ? top_launch<bf16_t>(p, stream) : top_launch<float>(p, stream);
}

}  // namespace spec
