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
// request's history once and keeps one 32-bit word per entry of the segment in shared
// memory:
//     bit 31 in the prompt | bits 20..30 bias slot + 1 | bits 0..19 count
// and one bit per entry that says whether the word is non-zero.  Rows are then streamed:
// a 16-byte word of logits whose bits are all clear (nearly all of them) only takes the
// temperature and the mask.  Between rows the next block token is added to the counts,
// so a history is scanned once per segment and not once per row.
#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kProcThreads = 256;
constexpr uint32_t kCountBits = 20, kCountMask = (1u << kCountBits) - 1u;
constexpr uint32_t kSlotMask = 0x7ffu, kInPrompt = 0x80000000u;

// Bits [e, e + 32) of a bit string, e >= 0 (one word past the end may be read).
__device__ __forceinline__ uint32_t bits_at(const uint32_t* w, int e) {
    return __funnelshift_r(w[e >> 5], w[(e >> 5) + 1], e & 31);
}

template <typename T>
__global__ void __launch_bounds__(kProcThreads) process_kernel(ProcessParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    extern __shared__ __align__(16) uint32_t s_proc[];
    uint32_t* s_state = s_proc;              // [seg]
    uint32_t* s_bits = s_proc + p.seg;       // [seg / 32 + 1]
    const int b = blockIdx.x / (p.n_seg * p.n_row_split);
    const int rem = blockIdx.x - b * (p.n_seg * p.n_row_split);
    const int rs = rem / p.n_seg, sg = rem - rs * p.n_seg;
    const int c0 = sg * p.seg;
    const int len = min(p.seg, p.V - c0);
    const int j0 = (int)((long)p.R * rs / p.n_row_split), j1 = (int)((long)p.R * (rs + 1) / p.n_row_split);
    const int tid = threadIdx.x;
    const bool report = sg == 0 && rs == 0;   // one CTA per request raises its flags

    const float rep = p.repetition ? p.repetition[b] : 1.0f;
    const float freq = p.frequency ? p.frequency[b] : 0.0f;
    const float pres = p.presence ? p.presence[b] : 0.0f;
    const float temp = p.temperature ? p.temperature[b] : 1.0f;
    const bool valid = rep > 0.0f && rep < INFINITY && temp > 0.0f && temp < INFINITY && fabsf(freq) < INFINITY &&
                       fabsf(pres) < INFINITY;
    int n = p.lengths ? p.lengths[b] : p.Lmax, m = p.prompt_lengths ? p.prompt_lengths[b] : 0;
    bool bad_token = n < 0 || n > p.Lmax || m < 0 || m > n;
    n = max(0, min(n, p.Lmax));
    m = max(0, min(m, n));
    const float rinv = 1.0f / rep, tinv = 1.0f / temp;

    for (int i = tid; i < p.seg; i += kProcThreads) s_state[i] = 0u;
    __syncthreads();
    if (p.nb > 0) {
        for (int i = tid; i < p.nb; i += kProcThreads) {
            const int id = p.bias_ids[(long)b * p.nb + i];
            if ((unsigned)(id - c0) < (unsigned)len) atomicMax(&s_state[id - c0], (uint32_t)(i + 1) << kCountBits);
            bad_token |= id < -1 || id >= p.V;
        }
        __syncthreads();
    }
    const int32_t* hist = p.history + (long)b * p.Lmax;
    for (int i = tid; i < n; i += kProcThreads) {
        const int t = hist[i];
        if ((unsigned)(t - c0) < (unsigned)len) {
            if (i < m) atomicOr(&s_state[t - c0], kInPrompt);
            else atomicAdd(&s_state[t - c0], 1u);
        }
        bad_token |= (unsigned)t >= (unsigned)p.V;
    }
    const int32_t* blk = p.block + (long)b * (p.R - 1);
    for (int i = tid; i < p.R - 1 && p.block; i += kProcThreads) {
        const int t = blk[i];
        if (i < j0 && (unsigned)(t - c0) < (unsigned)len) atomicAdd(&s_state[t - c0], 1u);
        bad_token |= (unsigned)t >= (unsigned)p.V;
    }
    if (report && bad_token) atomicOr(p.status, SPEC_DEV_TOKEN);
    if (report && !valid && tid == 0) atomicOr(p.status, SPEC_DEV_NONFINITE);
    __syncthreads();
    for (int i = tid; i < p.seg; i += kProcThreads) {   // seg is a multiple of kProcThreads
        const unsigned w = __ballot_sync(0xffffffffu, s_state[i] != 0u);
        if ((tid & 31) == 0) s_bits[i >> 5] = w;
    }
    if (tid == 0) s_bits[p.seg >> 5] = 0u;
    __syncthreads();

    for (int j = j0; j < j1; ++j) {
        if (j > j0 && p.block) {
            __syncthreads();   // row j - 1 has been read
            const int t = blk[j - 1];
            if (tid == 0 && (unsigned)(t - c0) < (unsigned)len) {
                s_state[t - c0] += 1u;
                s_bits[(t - c0) >> 5] |= 1u << ((t - c0) & 31);
            }
            __syncthreads();
        }
        const long row = (long)b * p.R + j;
        const RowWords<T> in(reinterpret_cast<const T*>(p.logits) + row * p.ld + c0, len);
        T* out = reinterpret_cast<T*>(p.out) + row * p.ld + c0;
        const uint32_t* mask =
            p.mask ? p.mask + ((p.mask_rows == 1 ? (long)b : row) * p.mask_words) + (c0 >> 5) : nullptr;
        const int mask_left = p.mask_words - (c0 >> 5);   // words from the segment's first
        for (int i = tid; i < in.n; i += kProcThreads) {
            const int e = in.entry(i);
            uint4 w = in.load(i);
            const int e0 = max(e, 0);
            // bit k of `touched` and `allowed` is entry e0 + k
            uint32_t touched = bits_at(s_bits, e0);
            uint32_t allowed = 0xffffffffu;
            if (mask) {
                const int mw = e0 >> 5;
                const uint32_t lo = __ldg(mask + mw);
                const uint32_t hi = mw + 1 < mask_left ? __ldg(mask + mw + 1) : 0u;
                allowed = __funnelshift_r(lo, hi, e0 & 31);
            }
            touched <<= e0 - e;
            allowed <<= e0 - e;
            float y[E];
#pragma unroll
            for (int k = 0; k < E; ++k) {
                float x = word_entry<T>(w, k);
                if ((touched >> k) & 1u && e + k >= 0 && e + k < len) {
                    const uint32_t st = s_state[e + k];
                    const uint32_t c = st & kCountMask, slot = (st >> kCountBits) & kSlotMask;
                    if (st & (kInPrompt | kCountMask)) x = x > 0.0f ? x * rinv : x * rep;
                    x -= fmaf(freq, (float)c, c ? pres : 0.0f);
                    if (slot) x += p.bias_values[(long)b * p.nb + slot - 1];
                }
                x *= tinv;
                if (!valid) x = NAN;
                y[k] = (allowed >> k) & 1u ? x : -INFINITY;
            }
            w = word_of<T>(y);
            in.store(out, i, w);
        }
    }
}

cudaError_t process_launch(ProcessParams p, cudaStream_t stream) {
    p.seg = 8192;
    p.n_seg = (p.V + p.seg - 1) / p.seg;
    p.n_row_split = 1;
    const size_t smem = ((size_t)p.seg + p.seg / 32 + 1) * sizeof(uint32_t);
    const long grid = (long)p.B * p.n_seg * p.n_row_split;
    if (grid > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    if (p.dtype == SPEC_BF16) process_kernel<bf16_t><<<(unsigned)grid, kProcThreads, smem, stream>>>(p);
    else process_kernel<float><<<(unsigned)grid, kProcThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace spec
