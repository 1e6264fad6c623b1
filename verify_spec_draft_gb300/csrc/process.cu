// process.cu - penalties, biases, temperature and grammar masks on the logits rows of a
// block (spec_process_logits).
//
// For request b with history h[0:n] (prompt h[0:m]) and block tokens x_1.., row j sees
// the context h[0:n] ++ x_1..x_j.  With c the occurrences of v in the generated part and
// seen(v) = c > 0 or v in the prompt,
//     y = l;  seen: y = y > 0 ? y / rho : y * rho;  y -= freq * c + pres * [c > 0];
//     y += bias(v);  y /= T;  y = -inf where the row's mask bit is 0.
//
// A CTA owns a segment of the vocabulary for some rows of one request.  It scans the
// request's history once, counting in shared memory with one 32-bit word per entry of the
// segment,
//     bit 31 in the prompt | bits 20..30 bias slot + 1 | bits 0..19 count,
// and then replaces each word by what the entry gets added, A = (bias - penalty) / T, with
// one bit per entry for "has something on it" and one for "seen".  Rows are then streamed:
// a 16-byte word of logits whose first bits are all clear (nearly all of them) only takes
// the temperature and the mask, the others one FFMA per entry, l * (1/T, rho/T or 1/(rho T))
// + A.  Between rows the next block token's entry is renewed, so a history is scanned once
// per segment and not once per row.
//
// Bound: bytes (each logit read and written once, a bit of mask), then instructions.  32 requests
// of 8 rows of 248,320 bf16 with histories of 8192, masks and 300 biases take 51 us of GPU time,
// 5.15 TB/s of what has to move and 77 % of a copy's rate; 48 M warp instructions keep the
// issue slots 72 % busy meanwhile.  Batches of 2 or 3 words take 57 and 59, entries touched one at
// a time instead of by whole words 55.  Against earlier stages of the kernel: one pass per row
// (every row's own counts) took 90; two batches of words in turn, not one requested ahead,
// changed nothing at 62.
#include <float.h>

#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kProcThreads = 256;
constexpr int kProcOcc = 4;   // CTAs per SM (the step above: 3 take 58 us, 5 take 63, 6 take 78)
constexpr uint32_t kCountBits = 20, kCountMask = (1u << kCountBits) - 1u;
constexpr uint32_t kSlotMask = 0x7ffu, kInPrompt = 0x80000000u;

// The kernel's shared memory: a word per entry of the segment, two strings of a bit per entry
// (each with eight words of room before it, kProcRoom), and for the block's tokens the
// token, its count and its bias.
constexpr int kProcRoom = 8;
__host__ __device__ constexpr int process_words(int seg) { return seg + 2 * (seg / 32) + 4 * kProcRoom; }
__host__ __device__ constexpr size_t process_smem(int seg) {
    return ((size_t)process_words(seg) + 3 * SPEC_MAX_GAMMA) * sizeof(uint32_t);
}

constexpr int kProcBatch = 4;   // words a thread holds while it waits for the ones behind

// One batch of a row: the words kProcThreads apart from word i0 + tid, and their mask words as
// they were loaded (nothing here waits for a load).
template <typename T, bool ALIGNED>
struct ProcBatch {
    uint4 w[kProcBatch];
    uint32_t mask[kProcBatch];
    __device__ __forceinline__ void load(const SegWords<T, ALIGNED>& in, const uint32_t* m, int mask_left, int i0) {
#pragma unroll
        for (int q = 0; q < kProcBatch; ++q) {
            const int i = i0 + q * kProcThreads + (int)threadIdx.x;
            if (i < in.n()) w[q] = in.load(i);
        }
        if (m) {
#pragma unroll
            for (int q = 0; q < kProcBatch; ++q) {
                const int i = i0 + q * kProcThreads + (int)threadIdx.x;
                if (i < in.n()) mask[q] = in.mask_word(m, mask_left, i);
            }
        }
    }
};

// A word's entries times f, rounded to T.
template <typename T>
__device__ __forceinline__ uint4 word_scaled(const uint4& w, float f) {
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[4];
    const f2x ff = f2_pack(f, f);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float2 y = f2_unpack(f2_mul(bf2_widen(h[r]), ff));
            o[r] = pack_bf16x2(y.x, y.y);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = __float_as_uint(__uint_as_float(h[r]) * f);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
// -inf where the word's bit is clear.
template <typename T>
__device__ __forceinline__ uint4 word_masked(const uint4& w, uint32_t allowed) {
    uint32_t h[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            // bits 2r and 2r + 1 to bits 15 and 31, then each over its half word
            const uint32_t v = allowed * ((1u << (15 - 2 * r)) | (1u << (30 - 2 * r)));
            uint32_t m;   // bytes 1 and 3 by their top bits (prmt's sign replication), twice each
            asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(m) : "r"(v));
            h[r] = (h[r] & m) | (NegInf<T>::word & ~m);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = (allowed >> r) & 1u ? h[r] : NegInf<T>::word;
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kProcThreads, kProcOcc) process_kernel(ProcessParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    extern __shared__ __align__(16) uint32_t s_proc[];
    uint32_t* s_state = s_proc + kProcRoom;                                // [seg]
    float* s_add = reinterpret_cast<float*>(s_state);                      // the same words, later
    uint32_t* s_bits = s_state + p.seg + kProcRoom;                        // [seg / 32] has something
    uint32_t* s_seen = s_bits + p.seg / 32 + kProcRoom;                    // [seg / 32]
    int32_t* s_blk = reinterpret_cast<int32_t*>(s_proc + process_words(p.seg));   // [R - 1] tokens
    int32_t* s_cnt = s_blk + SPEC_MAX_GAMMA;                               // [R - 1] counts once drafted
    float* s_bias = reinterpret_cast<float*>(s_cnt + SPEC_MAX_GAMMA);      // [R - 1]
    // segment by segment: the first ones, where frequent tokens tend to be, start first
    const int per_seg = p.B * p.n_row_split;
    const int sg = blockIdx.x / per_seg, rem = blockIdx.x - sg * per_seg;
    const int b = rem / p.n_row_split, rs = rem - b * p.n_row_split;
    const int c0 = sg * p.seg;
    const int len = min(p.seg, p.V - c0);
    const int j0 = rs * p.rows_per_cta, j1 = min(p.R, j0 + p.rows_per_cta);
    const int tid = threadIdx.x;
    const bool report = sg == 0 && rs == 0;   // one CTA per request raises its flags

    const int mask_left = p.mask_words - (c0 >> 5);   // words from the segment's first
    auto row_at = [&](int j) {
        return SegWords<T, ALIGNED>(reinterpret_cast<const T*>(p.logits) + ((long)b * p.R + j) * p.ld + c0, len);
    };
    auto mask_at = [&](int j) -> const uint32_t* {
        if (!p.mask) return nullptr;
        return p.mask + (p.mask_rows == 1 ? (long)b : (long)b * p.R + j) * p.mask_words + (c0 >> 5);
    };
    // the first batch is on its way while the history is scanned
    ProcBatch<T, ALIGNED> cur, nxt;
    cur.load(row_at(j0), mask_at(j0), mask_left, 0);

    const float rep = p.repetition ? p.repetition[b] : 1.0f;
    const float freq = p.frequency ? p.frequency[b] : 0.0f;
    const float pres = p.presence ? p.presence[b] : 0.0f;
    const float temp = p.temperature ? p.temperature[b] : 1.0f;
    int n = p.lengths ? p.lengths[b] : p.Lmax, m = p.prompt_lengths ? p.prompt_lengths[b] : 0;
    bool bad_token = n < 0 || n > p.Lmax || m < 0 || m > n;
    n = max(0, min(n, p.Lmax));
    m = max(0, min(m, n));

    // words and bits, 16 bytes at a time
    for (int i = tid; i < process_words(p.seg) / 4; i += kProcThreads)
        reinterpret_cast<uint4*>(s_proc)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.block && tid < p.R - 1) s_blk[tid] = p.block[(long)b * (p.R - 1) + tid];
    __syncthreads();
    auto mark = [&](int at) { atomicOr(&s_bits[at >> 5], 1u << (at & 31)); };
    if (p.nb > 0) {
        for (int i = tid; i < p.nb; i += kProcThreads) {
            const int id = p.bias_ids[(long)b * p.nb + i];
            if ((unsigned)(id - c0) < (unsigned)len) {
                atomicMax(&s_state[id - c0], (uint32_t)(i + 1) << kCountBits);
                mark(id - c0);
            }
            bad_token |= id < -1 || id >= p.V;
        }
        __syncthreads();
    }
    auto count = [&](int t, int i) {
        if ((unsigned)(t - c0) < (unsigned)len) {
            if (i < m) atomicOr(&s_state[t - c0], kInPrompt);
            else atomicAdd(&s_state[t - c0], 1u);
            mark(t - c0);
            atomicOr(&s_seen[(t - c0) >> 5], 1u << ((t - c0) & 31));
        }
        bad_token |= (unsigned)t >= (unsigned)p.V;
    };
    const int32_t* hist = p.history + (long)b * p.Lmax;
    const int n4 = p.hist_vec ? n / 4 : 0;   // whole 16-byte words of tokens
    unsigned worst = 0u;   // of the tokens, for the CTA that reports
#pragma unroll 4
    for (int i = tid; i < n4; i += kProcThreads) {
        const uint4 t = __ldg(reinterpret_cast<const uint4*>(hist) + i);
        if (report) worst = max(max(worst, max(t.x, t.y)), max(t.z, t.w));
        // four tokens at once: hardly any is in the segment
        if (min(min(t.x - c0, t.y - c0), min(t.z - c0, t.w - c0)) >= (unsigned)len) continue;
        count((int)t.x, 4 * i);
        count((int)t.y, 4 * i + 1);
        count((int)t.z, 4 * i + 2);
        count((int)t.w, 4 * i + 3);
    }
    bad_token |= worst >= (unsigned)p.V;
    for (int i = 4 * n4 + tid; i < n; i += kProcThreads) count(__ldg(hist + i), i);
    if (p.block && tid < p.R - 1) {
        if (tid < j0) count(s_blk[tid], p.Lmax);   // drafted before this CTA's first row
        else bad_token |= (unsigned)s_blk[tid] >= (unsigned)p.V;
    }
    float tinv = 1.0f / temp, f_pos = tinv / rep, f_neg = tinv * rep;   // the latter a seen entry's, by its sign
    // the factors are normal numbers: a logit of 0 or -inf stays what it is
    const float least = fminf(tinv, fminf(f_pos, f_neg)), most = fmaxf(tinv, fmaxf(f_pos, f_neg));
    const bool valid = rep > 0.0f && rep < INFINITY && temp > 0.0f && temp < INFINITY && least >= FLT_MIN &&
                       most <= FLT_MAX && fabsf(freq) < INFINITY && fabsf(pres) < INFINITY;
    if (report && bad_token) atomicOr(p.status, SPEC_DEV_TOKEN);
    if (report && !valid && tid == 0) atomicOr(p.status, SPEC_DEV_NONFINITE);
    if (!valid) tinv = f_pos = f_neg = NAN;
    __syncthreads();
    auto bias_of = [&](uint32_t st) {
        const uint32_t slot = (st >> kCountBits) & kSlotMask;
        return slot ? __ldg(p.bias_values + (long)b * p.nb + slot - 1) : 0.0f;
    };
    if (p.block && tid >= j0 && tid < j1 - 1 && (unsigned)(s_blk[tid] - c0) < (unsigned)len) {
        const uint32_t st = s_state[s_blk[tid] - c0];
        int c = (int)(st & kCountMask) + 1;
        for (int i = j0; i < tid; ++i) c += s_blk[i] == s_blk[tid] ? 1 : 0;
        s_cnt[tid] = c;
        s_bias[tid] = bias_of(st);
    }
    __syncthreads();
    for (int i = tid; i < p.seg / 32; i += kProcThreads)
        for (uint32_t w = s_bits[i]; w; w &= w - 1u) {
            const int at = i * 32 + __ffs(w) - 1;
            const uint32_t st = s_state[at], c = st & kCountMask;
            s_add[at] = (bias_of(st) - fmaf(freq, (float)c, c ? pres : 0.0f)) * tinv;
        }
    __syncthreads();

    for (int j = j0; j < j1; ++j) {
        if (j > j0 && p.block) {
            const int at = s_blk[j - 1] - c0;
            if ((unsigned)at < (unsigned)len) {   // the same for every thread
                __syncthreads();                  // row j - 1 has been read
                if (tid == 0) {
                    s_add[at] = (s_bias[j - 1] - fmaf(freq, (float)s_cnt[j - 1], pres)) * tinv;
                    s_bits[at >> 5] |= 1u << (at & 31);
                    s_seen[at >> 5] |= 1u << (at & 31);
                }
                __syncthreads();
            }
        }
        const SegWords<T, ALIGNED> in = row_at(j);
        T* out = reinterpret_cast<T*>(p.out) + ((long)b * p.R + j) * p.ld + c0;
        for (int i0 = 0; i0 < in.n(); i0 += kProcThreads * kProcBatch) {
            // the batch behind: of this row, or the next row's first
            if (i0 + kProcThreads * kProcBatch < in.n()) nxt.load(in, mask_at(j), mask_left, i0 + kProcThreads * kProcBatch);
            else if (j + 1 < j1) nxt.load(row_at(j + 1), mask_at(j + 1), mask_left, 0);
#pragma unroll
            for (int q = 0; q < kProcBatch; ++q) {
                const int i = i0 + q * kProcThreads + tid;
                if (i >= in.n()) break;
                uint4 o;
                if (in.bits(s_bits, i)) {
                    const uint32_t seen = in.bits(s_seen, i);
                    float add[E], y[E];
                    in.floats(s_add, i, add);
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const float x = word_entry<T>(cur.w[q], k);
                        y[k] = fmaf(x, (seen >> k) & 1u ? (x > 0.0f ? f_pos : f_neg) : tinv, add[k]);
                    }
                    o = word_of<T>(y);
                } else {
                    o = tinv == 1.0f ? cur.w[q] : word_scaled<T>(cur.w[q], tinv);
                }
                if (p.mask) o = word_masked<T>(o, in.allowed(cur.mask[q], i));
                in.store(out, i, o);
            }
            cur = nxt;
        }
    }
}

// Work split.  A CTA takes a segment of the vocabulary for r rows of a request.  In units of the
// time in which a resident CTA streams one word while all slots are taken (3.3 ns), it costs
//   to begin    1200, and a 14th per token of history, half per bias, a 36th per entry cleared,
//   a row       its words, 400 at least (a row's loads take that long, however few) and 110
//               for every batch of words behind the first, or less of them where slots
//               stay empty: down to three tenths.
// CTAs beyond the slots run in further waves, whose beginnings mostly hide behind the streams
// of other CTAs.  The split of least cost is taken; measured against all splits at eight
// sizes, it came within 7 percent of the best.
static long process_cost(const ProcessParams& p, int E, long slots, int r, long n, int* seg_out) {
    const int seg = (int)((p.V + n - 1) / n + 127) / 128 * 128;
    const long ctas = (long)((p.V + seg - 1) / seg) * ((p.R + r - 1) / r) * p.B;
    const long words = seg / E + 110 * ((seg / E - 1) / (kProcBatch * kProcThreads));
    const long waves = (ctas + slots - 1) / slots, last = ctas - (waves - 1) * slots;
    const long begin = 1200 + p.Lmax / 14 + p.nb / 2 + seg / 36;
    long thin = words * last / slots;
    if (thin < words * 3 / 10) thin = words * 3 / 10;
    *seg_out = seg;
    return begin + begin * 35 / 100 * (waves - 1) + r * ((waves - 1) * (words > 400 ? words : 400) + (thin > 400 ? thin : 400));
}

cudaError_t process_launch(ProcessParams p, cudaStream_t stream) {
    const int E = p.dtype == SPEC_BF16 ? 8 : 4;
    constexpr int kMaxSeg = 8832;   // 37 KB of shared memory; larger ones leave no L1 (serving step 56 us, not 51)
    static_assert(process_smem(kMaxSeg) <= 48 * 1024, "what a kernel gets without being asked for more");
    const long slots = (long)device_sm_count() * kProcOcc;
    const long least = (p.V + kMaxSeg - 1) / kMaxSeg;
    const long most = (p.V + 128 * E - 1) / (128 * E) > least ? (p.V + 128 * E - 1) / (128 * E) : least;
    long best = -1;
    for (int r = 1;; r = 2 * r < p.R ? 2 * r : p.R) {
        const long per = (long)p.B * ((p.R + r - 1) / r);
        for (int waves = 1; waves <= 3; ++waves) {
            long n = slots * waves / per;
            n = n < least ? least : (n > most ? most : n);
            int seg;
            const long cost = process_cost(p, E, slots, r, n, &seg);
            if (best < 0 || cost < best) {
                best = cost;
                p.seg = seg;
                p.rows_per_cta = r;
            }
        }
        if (r == p.R) break;
    }
    p.n_seg = (p.V + p.seg - 1) / p.seg;
    p.n_row_split = (p.R + p.rows_per_cta - 1) / p.rows_per_cta;
    p.hist_vec = p.Lmax % 4 == 0 && (reinterpret_cast<uintptr_t>(p.history) & 15u) == 0;
    const size_t smem = process_smem(p.seg);
    const long grid = (long)p.B * p.n_seg * p.n_row_split;
    if (grid > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    // rows of whole words move without tests for their ends: 51 us where the other kernel takes
    // 78 on the same rows
    const bool aligned = p.ld % E == 0 && p.V % E == 0;
    const void* kern = p.dtype == SPEC_BF16
                           ? (aligned ? (const void*)process_kernel<bf16_t, true> : (const void*)process_kernel<bf16_t, false>)
                           : (aligned ? (const void*)process_kernel<float, true> : (const void*)process_kernel<float, false>);
    void* args[] = {&p};
    return cudaLaunchKernel(kern, dim3((unsigned)grid), dim3(kProcThreads), args, smem, stream);
}

}  // namespace spec
