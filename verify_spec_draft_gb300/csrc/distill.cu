// distill.cu - distillation of a drafter's rows from a teacher's top logits
// (spec_distill): the loss and, on request, its gradient.
//
// A row's teacher is a distribution over K + 1 buckets: its K named entries and one for
// the rest of the vocabulary, p = softmax(a_1/t, .., a_K/t, a_T).  The student's row gives
// q = softmax(z/t), the named entries' q_k and the rest's q_T.  Then
//     L       = sum_k p_k ln(p_k / q_k) + p_T ln(p_T / q_T)
//     dL/dz_v = (q_v - p_k) / t             v named by k
//             = q_v (1 - p_T / q_T) / t     otherwise
// q_T is summed over the entries that no id names, never formed as 1 - sum q_k, so a rest
// of 1e-9 still has its logarithm.
//
// Weights and sums are taken relative to a maximum, and logarithms of p and q are differences
// from the two maxima, so the loss keeps float32's absolute accuracy whatever the logits'
// offset, and its digits where the named entries have little mass (row_ends).
#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kDistThreads = 128;
constexpr int kDistWarps = kDistThreads / 32;
constexpr int kDistWords = 12;                              // words a thread holds
constexpr int kDistPiece = kDistThreads * kDistWords;      // words of a CTA

__host__ __device__ inline int distill_pieces(int V, int elt_bytes) {
    const int E = 16 / elt_bytes;
    return ((V + 2 * E - 2) / E + kDistPiece - 1) / kDistPiece;
}

// Pairs (m, s): the maximum of some entries and the sum of their weights relative to it
// (row_words.cuh); empty: (-inf, 0).  NaN shows in m.
__device__ __forceinline__ float pair_weight(float2 v, float m, float c) {   // v's sum relative to m >= v.x
    return v.x == -INFINITY ? 0.0f : v.y * ex2(ref_rel(v.x, m, c));
}
__device__ __forceinline__ float2 pair_merge(float2 a, float2 b, float c) {
    const float m = f_max_nan(a.x, b.x);
    return make_float2(m, pair_weight(a, m, c) + pair_weight(b, m, c));
}
// Over the N lanes that differ in their low bits.
template <int N>
__device__ __forceinline__ float lanes_max_nan(float m) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) m = f_max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
template <int N>
__device__ __forceinline__ float lanes_sum(float s) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
template <int N>
__device__ __forceinline__ float2 pair_lanes(float2 v, float c) {
    const float m = N == 32 ? warp_max_nan(v.x) : lanes_max_nan<N>(v.x);
    return make_float2(m, lanes_sum<N>(pair_weight(v, m, c)));
}
// The pair of one entry per lane.
__device__ __forceinline__ float2 pair_entries(float x, float c) {
    const float m = warp_max_nan(x);
    return make_float2(m, lanes_sum<32>(x == -INFINITY ? 0.0f : ex2(ref_rel(x, m, c))));
}
constexpr float kMaxFloat = 3.402823466e38f;
constexpr uint32_t kBadToken = 0x7fc0dead;   // a NaN that says: an id is listed twice

// What the rows' ends share.  (M, Z): the student's pair, (mT, sT) that of its unnamed entries;
// amax: the teacher's largest named logit; top: the larger of it over t and the rest's aT; lag: how
// far amax / t lies below that; e, eT: the weights of the named entries and of the rest against
// top, P = e + eT; f the student's named weight against M.  Named entries are taken from
// amax before the scaling, so that their shares do not depend on how far from zero the teacher's
// logits are; amax / t itself, which only a rest is compared with, stops at the largest float.
//
// The share of the rest that the student has too much is
//     q_T - p_T = f_T / Z - e_T / P = (f_T e - e_T f) / (Z P),    f_T = sT 2^((mT - M) c),
// where the rest's own share is left out: with little named mass both shares are nearly 1,
// and their difference would keep none of its digits.  G is that without (sT / (Z P)).  The
// rest's part of the loss, p_T (ln p_T - ln q_T) = -p_T ln(1 + (q_T - p_T) / p_T), goes by it
// too, unless the shares are far apart: then the logarithms are taken one by one, for f_T may
// be too small for a float.
struct RowEnds { float M, Z, mT, sT, amax, top, lag, e, eT, P, G; };
__device__ __forceinline__ RowEnds row_ends(float2 T2, float2 N2, float2 teach, float aT, float c, float inv_t) {
    RowEnds r;
    const float2 A = pair_merge(T2, N2, c);
    r.M = A.x;
    r.Z = A.y;
    r.mT = T2.x;
    r.sT = T2.y;
    r.amax = teach.x;
    const float a = teach.x > -INFINITY ? fminf(fmaxf(teach.x * inv_t, -kMaxFloat), kMaxFloat) : teach.x;
    r.top = f_max_nan(a, aT);
    r.lag = a - r.top;
    r.e = teach.x > -INFINITY ? teach.y * __expf(r.lag) : 0.0f;
    r.eT = aT > -INFINITY ? __expf(aT - r.top) : 0.0f;
    r.P = r.e + r.eT;
    const float f = pair_weight(N2, A.x, c);
    r.G = T2.x > -INFINITY ? fmaf(ex2(ref_rel(T2.x, A.x, c)), r.e, -__fdividef(r.eT * f, T2.y)) : 0.0f;
    return r;
}
// ln of a named entry's weight against top
__device__ __forceinline__ float entry_log(const RowEnds& r, float a, float inv_t) {
    return a > -INFINITY ? fmaf(a - r.amax, inv_t, r.lag) : -INFINITY;
}
// p (M - x) / t, for a finite x so far below M that the difference overflows over t.  By halves, since
// M - x may overflow as well; the logarithms of the sums do not show beside it.
static __device__ __noinline__ float far_loss(float p, float M, float x, float inv_t) {
    return (2.0f * p * inv_t) * (0.5f * M - 0.5f * x);
}
__device__ __forceinline__ float entry_loss(const RowEnds& r, float a, float z, float inv_t) {
    const float lt = entry_log(r, a, inv_t), pk = __expf(lt) / r.P;
    if (!(pk > 0.0f)) return 0.0f;
    const float lz = (z - r.M) * inv_t;
    if (lz == -INFINITY && z > -INFINITY) return far_loss(pk, r.M, z, inv_t);
    return pk * ((lt - logf(r.P)) - (lz - logf(r.Z)));
}
__device__ __forceinline__ float rest_loss(const RowEnds& r, float aT, float inv_t) {
    const float pT = r.eT / r.P;
    if (!(pT > 0.0f)) return 0.0f;
    const bool some = r.mT > -INFINITY;
    const float d = some ? r.sT * r.G / (r.Z * r.eT) : -1.0f;
    if (fabsf(d) < 0.5f) return -pT * log1pf(d);
    const float lm = (r.mT - r.M) * inv_t;
    if (lm == -INFINITY && some) return far_loss(pT, r.M, r.mT, inv_t);
    const float lq = some ? lm + logf(r.sT) - logf(r.Z) : -INFINITY;
    return pT * (((aT - r.top) - logf(r.P)) - lq);
}

// ---------------------------------------------------------------------------------
// The loss alone: rows streamed once in pieces, (maximum, sum) of the entries that no id
// names per piece; the CTA that finishes a row's last piece forms the loss.  Bound by the
// rows' reads: 448 rows of 248,320 bf16 take 37.5 us, 5.9 TB/s, 89 % of a copy's rate.  128
// threads that hold twelve words each are small enough for a piece's end (one barrier, one
// record) to hide behind the other CTAs' loads and large enough for few ends: 256 threads take
// 43 us, 4 words 52, 16 words 45.
// ---------------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void distill_finish(const DistillParams& p, int row, float wt, int id);

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kDistThreads) distill_loss_kernel(DistillParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    __shared__ uint32_t s_named[kDistPiece * E / 32];
    __shared__ float2 s_run[kDistWarps];
    __shared__ uint32_t s_any[kDistWarps];   // bit q: something is named among a warp's q-th words
    __shared__ int s_twice;
    const int row = blockIdx.x / p.pieces, piece = blockIdx.x - row * p.pieces;
    const int tid = threadIdx.x, lane = tid & 31;
    const float wt = p.weight ? p.weight[row] : 1.0f;
    if (wt == 0.0f) {   // the row does not count and is not read
        if (piece == 0 && tid == 0) {
            p.loss_out[row] = 0.0f;
            if (p.lse_out) p.lse_out[row] = 0.0f;
        }
        return;
    }
    const SegWords<T, ALIGNED> in(reinterpret_cast<const T*>(p.student) + (long)row * p.ld, p.V);
    const int w0 = piece * kDistPiece, n = in.n();
    const uint32_t ninf = NegInf<T>::word;
    const int id = tid < p.K ? p.ids[(long)row * p.K + tid] : -1;
    uint4 w[kDistWords];
    if (w0 + kDistPiece <= n) {
#pragma unroll
        for (int q = 0; q < kDistWords; ++q) w[q] = in.load(w0 + q * kDistThreads + tid);
    } else {
#pragma unroll
        for (int q = 0; q < kDistWords; ++q) {
            const int i = w0 + q * kDistThreads + tid;
            w[q] = i < n ? in.load(i) : make_uint4(ninf, ninf, ninf, ninf);
        }
    }
    for (int i = tid; i < kDistPiece * E / 32; i += kDistThreads) s_named[i] = 0u;
    if (tid < kDistWarps) s_any[tid] = 0u;
    if (tid == 0) s_twice = 0;
    __syncthreads();
    const unsigned at = (unsigned)(id - in.entry(w0));
    if (id >= 0 && id < p.V && at < (unsigned)(kDistPiece * E)) {
        if ((atomicOr(&s_named[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1u) s_twice = 1;
        const int l = at / E;
        atomicOr(&s_any[(l / 32) % kDistWarps], 1u << (l / kDistThreads));
    }
    __syncthreads();
    const uint32_t any = s_any[tid >> 5];
    if (any) {
#pragma unroll
        for (int q = 0; q < kDistWords; ++q) {
            const int l = (q * kDistThreads + tid) * E;
            if ((any >> q) & 1u) w[q] = word_without<T>(w[q], (s_named[l >> 5] >> (l & 31)) & ((1u << E) - 1u));
        }
    }
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < kDistWords; ++q) m = f_max_nan(m, u4_max_nan<sizeof(T)>(w[q]));
    m = warp_max_nan(m);   // a NaN or +inf shows in the maximum
    const float s = warp_sum(words_sum<T, kDistWords>(w, m, p.scale));
    if (lane == 0) s_run[tid >> 5] = make_float2(m, s * ref_fix(m, p.scale));
    __syncthreads();
    if (tid < 32) {
        float2 t = pair_lanes<kDistWarps>(s_run[lane % kDistWarps], p.scale);
        if (s_twice) t.x = __uint_as_float(kBadToken);
        if (lane == 0) __stcg(&p.parts[(long)row * p.pieces + piece], t);
    }
    if (!last_block_done(&p.done[row], (unsigned)p.pieces)) return;
    if (tid == 0) p.done[row] = 0u;
    distill_finish<T>(p, row, wt, id);
}

template <typename T>
__device__ __forceinline__ void distill_finish(const DistillParams& p, int row, float wt, int id) {
    __shared__ float2 s_tail[kDistWarps], s_top[kDistWarps], s_teach[kDistWarps];
    __shared__ float s_loss[kDistWarps];
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float2 none = make_float2(-INFINITY, 0.0f);
    const bool there = id >= 0 && id < p.V;
    float z = -INFINITY, a = -INFINITY;
    if (there) {
        const T* src = reinterpret_cast<const T*>(p.student) + (long)row * p.ld + id;
        z = load_one(src);
        const long at = (long)row * p.K + tid;
        a = p.values_dtype == SPEC_BF16 ? to_float(reinterpret_cast<const bf16_t*>(p.values)[at])
                                        : reinterpret_cast<const float*>(p.values)[at];
    }
    const float aT = p.tail ? p.tail[row] : -INFINITY;
    int flag = id < -1 || id >= p.V ? 1 : 0;
    float2 t = none;
    for (int i = tid; i < p.pieces; i += kDistThreads) {
        const float2 v = __ldcg(&p.parts[(long)row * p.pieces + i]);
        if (__float_as_uint(v.x) == kBadToken) flag |= 1;
        t = pair_merge(t, v, p.scale);
    }
    if (!(a < INFINITY) || !(aT < INFINITY) || !(fabsf(wt) < INFINITY)) flag |= 2;
    if (tid == 0) s_flag = 0;
    t = pair_lanes<32>(t, p.scale);
    const float2 n = pair_entries(z, p.scale);
    const float2 y = pair_entries(a, p.scale);
    if (lane == 0) {
        s_tail[warp] = t;
        s_top[warp] = n;
        s_teach[warp] = y;
    }
    __syncthreads();
    if (flag) atomicOr(&s_flag, flag);
    // every warp puts the whole together
    const float2 T2 = pair_lanes<kDistWarps>(s_tail[lane % kDistWarps], p.scale);
    const float2 N2 = pair_lanes<kDistWarps>(s_top[lane % kDistWarps], p.scale);
    const RowEnds r = row_ends(T2, N2, pair_lanes<kDistWarps>(s_teach[lane % kDistWarps], p.scale), aT, p.scale, p.inv_t);
    float l = 0.0f;
    if (r.top > -INFINITY) {
        if (there) l = entry_loss(r, a, z, p.inv_t);
        if (tid == 0) l += rest_loss(r, aT, p.inv_t);
    }
    l = warp_sum(l);
    if (lane == 0) s_loss[warp] = l;
    __syncthreads();
    if (tid == 0) {
        const bool bad = s_flag || !(r.M < INFINITY) || r.M == -INFINITY;
        l = s_loss[0];
        for (int i = 1; i < kDistWarps; ++i) l += s_loss[i];
        p.loss_out[row] = bad ? NAN : l;
        if (p.lse_out) p.lse_out[row] = bad ? NAN : ref_log(r.M, r.Z, p.inv_t);
        if (s_flag & 1) atomicOr(p.status, SPEC_DEV_TOKEN);
        if ((s_flag & 2) || (bad && !(s_flag & 1))) atomicOr(p.status, SPEC_DEV_NONFINITE);
    }
}

// ---------------------------------------------------------------------------------
// Loss and gradient in one pass over the row.
//
// A row is split over a group of G CTAs; each holds its slice in shared memory from the read
// to the write of the gradient, so the logits are read once and the gradient is written once.
// The warps of a CTA have five jobs and meet at mbarriers only:
//   dense     A(i): the slice's (maximum, sum) over the entries that no id names;
//             B(i): every logit in the slot becomes its gradient, 2^(z c - m2) times one
//             factor.  In the order A(0) A(1) B(0) A(2) B(1) ..
//   take      one thread per teacher entry: takes the named logits out of the slice (-inf), the
//             teacher's row
//   exchange  posts the slice's statistics, waits for the other slices', forms the factor
//   fix       one thread per teacher entry: puts the named entries' gradients in after B(i),
//             then forms the loss
//   copies    slices in and out
// So the row behind is reduced while the statistics of the row before travel (2000 to 4000
// cycles on a loaded memory system, about as long as A and B), its named entries are out by
// then, and three or four slots keep one slice arriving and one leaving meanwhile.  With take
// and fix in the same warps, A(i + 2) waited for fix(i): 2000 rows of 20,000 bf16 took 48 us and
// not 42, today 40.
//
// The exchange: a record per CTA in global memory, each 64-bit word a value and a tag that no
// earlier row or call has used, so a word is valid when its tag is and nothing else has to
// be ordered.  A record's place is used again two exchanges later: a CTA that posts the
// (j + 1)th has seen every post of the jth, and each came after its CTA had read the
// (j - 1)th.  In place of the logits the gradient is safe for the same reason: a slice is
// written after every record of its row has arrived, and a record holds what was read.
//
// A wait that runs out sets SPEC_DEV_TIMEOUT and s_gave_up, before whatever the waiter hands on.
// From then on the CTA waits for nothing more, posts NaN, touches no slot, loads nothing more, and
// writes NaN for the rows that it has not written, once its loads in flight have landed.
//
// Bound by memory, a read and a write of each logit: 1792 rows of 248,320 bf16 take 297 to 320 us
// from one GPU to another.  One row in ten has weight 0 there and is written but not read, so that
// 1.69 GB move, at 5.3 to 5.7 TB/s, 79 to 85 % of a copy's rate.  What is missing is
// residency: with 210 KB of slices in an SM and 3.5 us a row, the slot that waits for the
// exchange is one of three that would otherwise load or store.  Short rows are bound by the
// steps from A(i) to B(i), 1.5 us a row.  For the 1792 rows, when they took 292 to 309, reading them
// twice took 392 us; slices in registers with the whole CTA waiting on the exchange 834; two
// CTAs per SM with three slots of 32 KB 335, three CTAs 372 to 427; four slots of 56 KB 345; the
// reduction and the gradient in separate warps 440; 256, 320 or 512 dense threads 2 to 5 % longer.
// ---------------------------------------------------------------------------------
constexpr int kFuseDense = 384;                            // threads of the dense warps
constexpr int kFuseNamed = SPEC_MAX_TEACHER;               // threads of either job on the entries
constexpr int kFuseThreads = kFuseDense + 2 * kFuseNamed + 64;   // and a warp each to exchange and to copy
constexpr int kDenseWarps = kFuseDense / 32, kNamedWarps = kFuseNamed / 32;
constexpr int kFuseOcc = 1;                                // CTAs per SM
constexpr int kFuseBatch = 4;                              // words a dense thread holds at once
constexpr int kFuseSlice = 4480;                           // most words of a slice (70 KB)
constexpr int kFuseRoom = 3 * kFuseSlice;                  // words of slices in shared memory
constexpr int kFuseRecord = 4;                             // words of a record
constexpr int kFuseRing = 2;                               // exchanges a record's place lasts
constexpr int kFuseMaxCtas = 512;

struct FuseHeader {
    unsigned epoch;    // tags up to here have been used
    unsigned exits;    // CTAs that have left (0 between calls)
    // 0 but in tests of a wait that runs out: how long one may take in us (0: kWaitLimitNs), and the
    // exchange, from 1 on, whose record the first CTA keeps back.
    unsigned patience, withheld;
    unsigned pad[60];
};

__device__ __forceinline__ void post_word(unsigned long long* p, float v, unsigned tag) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;"
                 :: "l"(p), "l"(((unsigned long long)tag << 32) | __float_as_uint(v)) : "memory");
}
__device__ __forceinline__ unsigned long long peek_word(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, unsigned bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                 :: "l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_s2g_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_s2g_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
template <int BAR>   // the warps of a job on the entries
__device__ __forceinline__ void named_sync() { asm volatile("bar.sync %0, %1;" :: "n"(BAR), "n"(kFuseNamed) : "memory"); }

__device__ __forceinline__ unsigned long long fuse_limit(const FuseHeader* h) {
    const unsigned us = *(const volatile unsigned*)&h->patience;
    return us ? us * 1000ull : kWaitLimitNs;
}
// The rest of a wait whose first try failed: false when it ran out, here or in another thread.  Out of
// line, as a dozen copies of it are instructions that the jobs' chains wait for.
static __device__ __noinline__ bool fuse_wait(uint64_t* bar, unsigned parity, unsigned* status, const FuseHeader* h,
                                              volatile int* gave_up) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    if (!*gave_up && mbar_wait(bar, parity, status, fuse_limit(h))) return true;
    *gave_up = 1;
    return false;
}

// What is known of a row once its slices' statistics are together.
struct FuseRow : RowEnds {
    float ref;        // R(mT).  Unnamed entries: gradient 2^(z c - ref) factor, beyond kRefNear 2^((z - mT) c) factor
    float factor;
    float wt, aT;     // the row's weight, the teacher's rest
    int skip, bad;
};
// What becomes of a named entry: the logits of student and teacher, its id and its place in
// the slice (-1: none).
struct FuseEntry { float z, a; int id, at; };

// The slice of a row that one CTA holds: words [0, n) of it, whole words [a, b).
template <typename T>
struct Slice {
    RowWords<T> in;
    int first, n, a, b;
    __device__ __forceinline__ Slice(const T* row, int V, int first_, int most) : in(row, V), first(first_) {
        n = max(0, min(in.n - first, most));
        a = n > 0 && !in.whole(first) ? 1 : 0;
        b = n > a && !in.whole(first + n - 1) ? n - 1 : max(n, a);
    }
};

template <typename T, int SLOTS>
__global__ void __launch_bounds__(kFuseThreads, kFuseOcc) distill_fused_kernel(DistillParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) uint8_t s_slots[];
    // full: a slice has arrived; ready: its named entries are out; reduced: A is done; stated:
    // the teacher's statistics are there; known: the row's FuseRow is; dense: B is done;
    // fixed: the named entries' gradients are in.  What comes back with its slot does so after
    // the slot's last user, fixed; what comes back two rows on (by parity) after known, which
    // `take` waits for.  So no waiter can miss a phase, and no shared word is written before
    // its readers are done.
    __shared__ __align__(8) uint64_t s_full[SLOTS], s_fixed[SLOTS], s_known[SLOTS], s_dense[SLOTS];
    __shared__ __align__(8) uint64_t s_ready[2], s_reduced[2], s_stated[2];
    __shared__ uint32_t s_bits[kFuseSlice * E / 32];         // the slice's entries named so far
    __shared__ float2 s_tail[2][kDenseWarps], s_top[2][kNamedWarps], s_teach[2][kNamedWarps];
    __shared__ float s_loss[2][kNamedWarps], s_wt[2], s_aT[2];
    __shared__ int s_flag[2], s_gave_up;
    __shared__ FuseRow s_row[SLOTS];
    __shared__ FuseEntry s_entry[SLOTS][kFuseNamed];
    const int tid = threadIdx.x, lane = tid & 31;
    const int group = blockIdx.x / p.group_size, rank = blockIdx.x - group * p.group_size;
    const int n_it = (p.rows - group + p.n_groups - 1) / p.n_groups;
    const float c = p.scale;
    const unsigned epoch = *(volatile unsigned*)&p.fuse->epoch;

    auto row_of = [&](int i) { return group + i * p.n_groups; };
    auto slice_of = [&](int i) {
        return Slice<T>(reinterpret_cast<const T*>(p.student) + (long)row_of(i) * p.ld, p.V, rank * p.slice, p.slice);
    };
    auto grad_of = [&](int i) { return reinterpret_cast<T*>(p.grad_out) + (long)row_of(i) * p.ld; };
    auto slot_of = [&](int i) { return reinterpret_cast<uint4*>(s_slots) + (size_t)(i % SLOTS) * p.slice; };

    if (tid == 0) {
        for (int q = 0; q < SLOTS; ++q) {
            mbar_init(&s_full[q], 1);
            mbar_init(&s_fixed[q], kFuseNamed);
            mbar_init(&s_known[q], 1);
            mbar_init(&s_dense[q], kDenseWarps);
        }
        for (int q = 0; q < 2; ++q) {
            mbar_init(&s_ready[q], kFuseNamed);
            mbar_init(&s_reduced[q], kDenseWarps);
            mbar_init(&s_stated[q], kNamedWarps);
            s_flag[q] = 0;
        }
        s_gave_up = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < kFuseSlice * E / 32; i += kFuseThreads) s_bits[i] = 0u;
    __syncthreads();
    auto gave_up = [&] { return *(volatile int*)&s_gave_up != 0; };
    bool dead = false;   // this thread's waits so far have not all ended well
    auto wait = [&](uint64_t* bar, int phase) {
        if (!dead && !mbar_try_wait(bar, phase & 1)) dead = !fuse_wait(bar, phase & 1, p.status, p.fuse, &s_gave_up);
    };

    if (tid < kFuseDense) {
        // ------------------------------------------------------------------ dense
        const int warp = tid >> 5;
        const f2x cc = f2_pack(c, c);
        for (int i = 0; i <= n_it; ++i) {
            if (i < n_it) {   // A(i)
                const int n = slice_of(i).n;
                const uint4* slot = slot_of(i);
                wait(&s_full[i % SLOTS], i / SLOTS);
                wait(&s_ready[i & 1], i >> 1);
                if (s_wt[i & 1] != 0.0f) {
                    float m = -INFINITY, s = 0.0f;
                    for (int l0 = 0; l0 < n; l0 += kFuseDense * kFuseBatch) {
                        uint4 w[kFuseBatch];
                        const uint32_t ninf = NegInf<T>::word;
                        float bm = -INFINITY;
#pragma unroll
                        for (int q = 0; q < kFuseBatch; ++q) {
                            const int l = l0 + q * kFuseDense + tid;
                            w[q] = l < n ? slot[l] : make_uint4(ninf, ninf, ninf, ninf);
                        }
#pragma unroll
                        for (int q = 0; q < kFuseBatch; ++q) bm = f_max_nan(bm, u4_max_nan<sizeof(T)>(w[q]));
                        // a thread's own running maximum; a batch of -inf adds nothing
                        bm = f_max_nan(bm, m);
                        if (bm != m) {
                            s = m == -INFINITY ? 0.0f : s * ex2(ref_step(m, bm, c));
                            m = bm;
                        }
                        s += words_sum<T, kFuseBatch>(w, m, c);
                    }
                    if (dead) m = NAN;
                    const float2 t = pair_lanes<32>(make_float2(m, s * ref_fix(m, c)), c);
                    if (lane == 0) s_tail[i & 1][warp] = t;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive1(&s_reduced[i & 1]);
            }
            if (i >= 1) {     // B(i - 1)
                const int j = i - 1, n = slice_of(j).n;
                uint4* slot = slot_of(j);
                wait(&s_known[j % SLOTS], j / SLOTS);
                const FuseRow& row = s_row[j % SLOTS];
                const float x = row.ref;
                if (dead) {
                    // the slot is not this row's
                } else if (row.skip) {
                    for (int l = tid; l < n; l += kFuseDense) slot[l] = make_uint4(0u, 0u, 0u, 0u);
                } else if (ref_near(x)) {
                    const f2x mm = f2_pack(-x, -x), ff = f2_pack(row.factor, row.factor);
#pragma unroll 4
                    for (int l = tid; l < n; l += kFuseDense) {
                        const uint4 w = slot[l];
                        float d[E];
#pragma unroll
                        for (int k = 0; k < E; k += 2) {
                            const float2 y = f2_unpack(f2_mul(
                                f2_ex2(f2_fma(f2_pack(word_entry<T>(w, k), word_entry<T>(w, k + 1)), cc, mm)), ff));
                            d[k] = y.x;
                            d[k + 1] = y.y;
                        }
                        slot[l] = word_of<T>(d);
                    }
                } else {   // the unnamed entries are far from zero
                    for (int l = tid; l < n; l += kFuseDense) {
                        const uint4 w = slot[l];
                        float d[E];
#pragma unroll
                        for (int k = 0; k < E; ++k) d[k] = ex2((word_entry<T>(w, k) - row.mT) * c) * row.factor;
                        slot[l] = word_of<T>(d);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&s_dense[j % SLOTS]);
            }
        }
    } else if (tid < kFuseDense + kFuseNamed) {
        // ------------------------------------------------------------------- take
        const int k = tid - kFuseDense, warp = k >> 5;
        // thread k's teacher entry of a row, the student's logit there (where it is known), and
        // what the row's entries share
        struct Entry { int id; float a, z; float wt, aT; };
        auto load = [&](int i, Entry& e) {
            e.id = -1;
            e.a = e.z = e.aT = -INFINITY;
            e.wt = 0.0f;
            if (i >= n_it) return;
            const int row = row_of(i);
            e.wt = p.weight ? p.weight[row] : 1.0f;
            if (p.tail) e.aT = p.tail[row];
            if (k >= p.K) return;
            const long at = (long)row * p.K + k;
            e.id = p.ids[at];
            e.a = p.values_dtype == SPEC_BF16 ? to_float(reinterpret_cast<const bf16_t*>(p.values)[at])
                                              : reinterpret_cast<const float*>(p.values)[at];
        };
        auto known_id = [&](const Entry& e) { return e.id >= 0 && e.id < p.V; };
        // slice 0 forms the loss, so it reads all of its row's named logits
        auto gather = [&](int i, Entry& e) {
            if (i >= n_it || rank != 0 || !known_id(e) || e.wt == 0.0f) return;
            const T* z = reinterpret_cast<const T*>(p.student) + (long)row_of(i) * p.ld + e.id;
            if (sizeof(T) == 2) e.z = to_float((bf16_t)*reinterpret_cast<const volatile unsigned short*>(z));
            else e.z = to_float(*reinterpret_cast<const volatile float*>(z));
        };
        Entry cur, nxt, far;
        load(0, cur);
        load(1, nxt);
        gather(0, cur);
        for (int i = 0; i < n_it; ++i) {
            const int par = i & 1;
            gather(i + 1, nxt);
            load(i + 2, far);
            named_sync<1>();   // the bits are clear again
            const Slice<T> sl = slice_of(i);
            const int in_slice = cur.id - sl.in.entry(sl.first);
            const int at = known_id(cur) && in_slice >= 0 && in_slice < sl.n * E ? in_slice : -1;
            int f = 0;
            if (at >= 0 && (atomicOr(&s_bits[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1u) f = 1;   // listed twice
            if (i >= 2) wait(&s_known[(i - 2) % SLOTS], (i - 2) / SLOTS);
            if (k == 0) {
                s_wt[par] = cur.wt;
                s_aT[par] = cur.aT;
            }
            wait(&s_full[i % SLOTS], i / SLOTS);
            if (!dead && at >= 0 && cur.wt != 0.0f) {
                T* x = reinterpret_cast<T*>(slot_of(i)) + at;
                cur.z = to_float(*x);
                *x = sizeof(T) == 2 ? (T)0xff80u : (T)-INFINITY;
            }
            mbar_arrive1(&s_ready[par]);
            s_entry[i % SLOTS][k] = {cur.z, cur.a, cur.id, at};
            if (cur.wt != 0.0f) {
                const float a = known_id(cur) ? cur.a : -INFINITY;
                const float2 t = pair_entries(a, c);
                const float2 z = pair_entries(rank == 0 ? cur.z : -INFINITY, c);
                if (lane == 0) {
                    s_teach[par][warp] = t;
                    s_top[par][warp] = z;
                }
                if (dead) f |= 4;
                if (rank == 0) {
                    f |= (cur.id < -1 || cur.id >= p.V) ? 1 : 0;
                    if (!(a < INFINITY) || !(cur.aT < INFINITY) || !(fabsf(cur.wt) < INFINITY)) f |= 2;
                }
                if (f) atomicOr(&s_flag[par], f);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(&s_stated[par]);
            named_sync<1>();   // every entry's bit has been looked at
            if (at >= 0) s_bits[at >> 5] = 0u;
            cur = nxt;
            nxt = far;
        }
    } else if (tid < kFuseDense + 2 * kFuseNamed) {
        // -------------------------------------------------------------------- fix
        const int k = tid - kFuseDense - kFuseNamed, warp = k >> 5;
        for (int i = 0; i < n_it; ++i) {
            const int row = row_of(i), par = i & 1;
            wait(&s_known[i % SLOTS], i / SLOTS);
            const FuseRow r = s_row[i % SLOTS];
            const FuseEntry e = s_entry[i % SLOTS][k];
            const bool taught = r.top > -INFINITY, named = e.id >= 0 && e.id < p.V;
            float d = 0.0f;
            if (!r.skip && e.at >= 0) {
                const float pk = taught ? __expf(entry_log(r, e.a, p.inv_t)) / r.P : 0.0f;
                d = r.bad ? NAN : (taught ? (ex2(ref_rel(e.z, r.M, c)) / r.Z - pk) * (r.wt * p.inv_t) : 0.0f);
            }
            wait(&s_dense[i % SLOTS], i / SLOTS);
            const bool lost = gave_up();   // then what was read above may be anything
            if (!lost && e.at >= 0 && !r.skip) {
                T* x = reinterpret_cast<T*>(slot_of(i)) + e.at;
                if (sizeof(T) == 2) *x = (T)__bfloat16_as_ushort(__float2bfloat16_rn(d));
                else *x = (T)d;
            }
            fence_proxy_async_smem();
            mbar_arrive1(&s_fixed[i % SLOTS]);
            if (rank != 0) continue;
            float l = 0.0f;   // the loss, behind what the slice waits for
            if (!lost && !r.skip && taught) {
                if (named) l = entry_loss(r, e.a, e.z, p.inv_t);
                if (k == 0) l += rest_loss(r, r.aT, p.inv_t);
            }
            l = warp_sum(l);
            if (lane == 0) s_loss[par][warp] = l;
            named_sync<2>();
            if (k == 0) {
                l = s_loss[par][0];
                for (int q = 1; q < kNamedWarps; ++q) l += s_loss[par][q];
                const bool bad = gave_up() || (!r.skip && r.bad);
                p.loss_out[row] = bad ? NAN : (r.skip ? 0.0f : l);
                if (p.lse_out) p.lse_out[row] = bad ? NAN : (r.skip ? 0.0f : ref_log(r.M, r.Z, p.inv_t));
            }
        }
    } else if (tid < kFuseDense + 2 * kFuseNamed + 32) {
        // --------------------------------------------------------------- exchange
        unsigned long long* recs = p.records + (size_t)group * kFuseRing * p.group_size * kFuseRecord;
        const float2 none = make_float2(-INFINITY, 0.0f);
        unsigned live = 0;       // exchanges so far: rows that count
        const unsigned withheld = *(volatile unsigned*)&p.fuse->withheld;
        for (int i = 0; i < n_it; ++i) {
            const int par = i & 1;
            wait(&s_stated[par], i >> 1);
            const float wt = s_wt[par], aT = s_aT[par];
            const bool skip = wt == 0.0f;
            // the teacher's named entries, the student's (slice 0 has them)
            const float2 tn = pair_lanes<4>(skip ? none : s_teach[par][lane & 3], c);
            const float2 nn = pair_lanes<4>(skip ? none : s_top[par][lane & 3], c);
            static_assert(kNamedWarps == 4 && kDenseWarps <= 16, "the lanes' layout");
            const int flag = s_flag[par];
            float2 T2 = none, N2 = none;
            bool token = false, late = false;
            wait(&s_reduced[par], i >> 1);
            if (!skip && p.group_size == 1) {   // nobody to exchange with
                T2 = pair_lanes<16>((lane & 15) < kDenseWarps ? s_tail[par][lane & 15] : none, c);
                if (flag || dead) T2.x = NAN;
                N2 = nn;
                token = flag & 1;
                late = dead;
            } else if (!skip) {
                unsigned long long* rec = recs + (size_t)(live % kFuseRing) * p.group_size * kFuseRecord;
                const unsigned tag = epoch + 1u + live;
                ++live;
                float2 t = pair_lanes<16>((lane & 15) < kDenseWarps ? s_tail[par][lane & 15] : none, c);
                if (flag || dead) t.x = flag & 1 ? __uint_as_float(kBadToken) : NAN;
                if (lane < (rank == 0 ? 4 : 2) && (live != withheld || blockIdx.x != 0))
                    post_word(rec + (size_t)rank * kFuseRecord + lane, lane == 0 ? t.x : (lane == 1 ? t.y : (lane == 2 ? nn.x : nn.y)), tag);
                const unsigned long long t0 = global_timer_ns();
                for (int r = lane; r < p.group_size; r += 32) {
                    unsigned long long v[kFuseRecord] = {0ull, 0ull, 0ull, 0ull};
                    const unsigned long long* src = rec + (size_t)r * kFuseRecord;
                    unsigned spins = 0;
                    while (true) {
                        bool here = true;
#pragma unroll
                        for (int q = 0; q < kFuseRecord; ++q)
                            if (q < 2 || r == 0) v[q] = peek_word(src + q);
#pragma unroll
                        for (int q = 0; q < kFuseRecord; ++q)
                            if (q < 2 || r == 0) here &= (unsigned)(v[q] >> 32) == tag;
                        if (here) break;
                        if (dead || late || (((++spins) & 63u) == 0 && global_timer_ns() - t0 > fuse_limit(p.fuse))) {
                            late = true;
                            break;
                        }
                    }
                    token |= (uint32_t)v[0] == kBadToken;
                    T2 = pair_merge(T2, make_float2(__uint_as_float((uint32_t)v[0]), __uint_as_float((uint32_t)v[1])), c);
                    if (r == 0) N2 = make_float2(__uint_as_float((uint32_t)v[2]), __uint_as_float((uint32_t)v[3]));
                }
                late = __any_sync(0xffffffffu, late);
                token = __any_sync(0xffffffffu, token);
                if (late) {
                    *(volatile int*)&s_gave_up = 1;
                    dead = true;
                }
                T2 = pair_lanes<32>(T2, c);
                N2.x = __shfl_sync(0xffffffffu, N2.x, 0);
                N2.y = __shfl_sync(0xffffffffu, N2.y, 0);
            }
            if (lane == 0) {
                FuseRow r;
                static_cast<RowEnds&>(r) = row_ends(T2, N2, skip ? none : tn, skip ? -INFINITY : aT, c, p.inv_t);
                const bool bad = !skip && (late || !(r.M < INFINITY) || r.M == -INFINITY);
                r.ref = r.mT > -INFINITY ? r.mT * c : 0.0f;
                r.factor = r.top > -INFINITY ? wt * p.inv_t * __fdividef(r.G, r.Z * r.P) * ref_fix(r.mT, c) : 0.0f;
                if (bad) r.factor = NAN;
                r.skip = skip;
                r.bad = bad;
                r.wt = wt;
                r.aT = aT;
                s_row[i % SLOTS] = r;
                s_flag[par] = 0;
                mbar_arrive1(&s_known[i % SLOTS]);
                unsigned raise = 0u;
                if (flag & 1) raise |= SPEC_DEV_TOKEN;
                if ((flag & 2) || (bad && rank == 0 && !token && !late)) raise |= SPEC_DEV_NONFINITE;
                if (late) raise |= SPEC_DEV_TIMEOUT;
                if (raise) atomicOr(p.status, raise);
            }
            __syncwarp();
        }
    } else {
        // ----------------------------------------------------------------- copies
        auto issue = [&](int i) {   // the warp: row i's slice on its way to its slot
            uint64_t* bar = &s_full[i % SLOTS];
            const Slice<T> sl = slice_of(i);
            const bool on = !(p.weight && p.weight[row_of(i)] == 0.0f);
            if (on && lane < 2) {   // the words that are not whole
                const int l = lane == 0 ? 0 : sl.b;
                if (lane == 0 ? sl.a > 0 : sl.b < sl.n) slot_of(i)[l] = sl.in.load(sl.first + l);
            }
            __syncwarp();
            if (lane == 0) {
                if (on && sl.a < sl.b) {
                    const unsigned bytes = (unsigned)(sl.b - sl.a) * 16u;
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_g2s(slot_of(i) + sl.a, sl.in.p + sl.in.entry(sl.first + sl.a), bytes, bar);
                } else {
                    mbar_arrive1(bar);
                }
            }
        };
        int i = 0;
        for (int q = 0; q < SLOTS && q < n_it; ++q) issue(q);
        for (; i < n_it; ++i) {
            wait(&s_fixed[i % SLOTS], i / SLOTS);
            if (__any_sync(0xffffffffu, gave_up())) break;
            const Slice<T> sl = slice_of(i);
            if (lane == 0 && sl.a < sl.b)
                bulk_s2g(grad_of(i) + sl.in.entry(sl.first + sl.a), slot_of(i) + sl.a, (unsigned)(sl.b - sl.a) * 16u);
            if (lane < 2) {
                const int l = lane == 0 ? 0 : sl.b;
                if (lane == 0 ? sl.a > 0 : sl.b < sl.n) sl.in.store(grad_of(i), sl.first + l, slot_of(i)[l]);
            }
            if (i + SLOTS < n_it) {
                if (lane == 0) bulk_s2g_wait_read();
                fence_proxy_async_smem();   // the words that were not whole, before the copy that may cover them
                __syncwarp();
                issue(i + SLOTS);
            }
        }
        if (i < n_it) {   // a wait has run out
            for (int q = i; q < i + SLOTS && q < n_it; ++q)
                mbar_wait(&s_full[q % SLOTS], (q / SLOTS) & 1, p.status, kWaitLimitNs);
            for (; i < n_it; ++i) {
                const Slice<T> sl = slice_of(i);
                const uint32_t nan = sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu;
                for (int l = lane; l < sl.n; l += 32) sl.in.store(grad_of(i), sl.first + l, make_uint4(nan, nan, nan, nan));
            }
        }
        if (lane == 0) {
            bulk_s2g_wait();
            // the last CTA to leave retires the call's tags: its slices' gradients are out, so
            // every record that it needed has been read
            const unsigned n = p.n_groups * p.group_size;
            if (atom_add_acq_rel(&p.fuse->exits, 1u) == n - 1u) {
                atomicExch(&p.fuse->exits, 0u);
                atomicExch(&p.fuse->epoch, epoch + (unsigned)((p.rows + p.n_groups - 1) / p.n_groups) + 1u);
            }
        }
    }
}

template <typename T>
static cudaError_t fused_launch(DistillParams p, cudaStream_t stream) {
    const int ctas = device_sm_count() * kFuseOcc < kFuseMaxCtas ? device_sm_count() * kFuseOcc : kFuseMaxCtas;
    const int words = (p.V + 2 * (16 / (int)sizeof(T)) - 2) / (16 / (int)sizeof(T));   // whatever the row's offset
    const int least = (words + kFuseSlice - 1) / kFuseSlice;
    if (least > ctas) return cudaErrorInvalidConfiguration;
    // as many rows at once as there are CTAs for, then the CTAs left over go to the groups,
    // down to a slice of one word per dense thread
    int groups = ctas / least;
    if (groups > p.rows) groups = p.rows;
    int size = ctas / groups;
    const int most = (words + kFuseDense - 1) / kFuseDense;
    if (size > most) size = most > least ? most : least;
    p.n_groups = groups;
    p.group_size = size;
    p.slice = (words + size - 1) / size;
    // a fourth slot where there is room for one: 1000 rows of 20,001 float32 took 41 us instead of
    // 43, 2000 of 20,000 bf16 39 instead of 42 (smaller slices for its sake cost more than it gives)
    const int slots = 4 * p.slice <= kFuseRoom ? 4 : 3;
    const void* kern = slots == 4 ? (const void*)distill_fused_kernel<T, 4> : (const void*)distill_fused_kernel<T, 3>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFuseRoom * 16);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    return cudaLaunchCooperativeKernel(kern, dim3(groups * size), dim3(kFuseThreads), args, (size_t)slots * p.slice * 16,
                                       stream);
}

constexpr size_t kFuseBytes = sizeof(FuseHeader) + sizeof(unsigned long long) * kFuseMaxCtas * kFuseRing * kFuseRecord;

size_t distill_workspace_bytes(int rows, int V) {
    return kWsHeaderBytes + align256(kFuseBytes) + align256((size_t)rows * sizeof(unsigned)) +
           (size_t)rows * distill_pieces(V, 4) * sizeof(float2);
}

template <typename T>
static cudaError_t distill_typed(DistillParams p, cudaStream_t stream) {
    if (p.grad_out) return fused_launch<T>(p, stream);
    p.pieces = distill_pieces(p.V, sizeof(T));
    const long grid = (long)p.rows * p.pieces;
    if (grid > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    if (SegWords<T, true>::fits(p.ld, p.V)) distill_loss_kernel<T, true><<<(unsigned)grid, kDistThreads, 0, stream>>>(p);
    else distill_loss_kernel<T, false><<<(unsigned)grid, kDistThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t distill_launch(DistillParams p, void* ws, cudaStream_t stream) {
    p.status = &reinterpret_cast<WsHeader*>(ws)->status;
    uint8_t* b = reinterpret_cast<uint8_t*>(ws) + kWsHeaderBytes;
    p.fuse = reinterpret_cast<FuseHeader*>(b);
    p.records = reinterpret_cast<unsigned long long*>(b + sizeof(FuseHeader));
    b += align256(kFuseBytes);
    p.done = reinterpret_cast<unsigned*>(b);
    p.parts = reinterpret_cast<float2*>(b + align256((size_t)p.rows * sizeof(unsigned)));
    return p.dtype == SPEC_BF16 ? distill_typed<bf16_t>(p, stream) : distill_typed<float>(p, stream);
}

}  // namespace spec
