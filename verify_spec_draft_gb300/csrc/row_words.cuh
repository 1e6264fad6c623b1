// row_words.cuh - rows of any length and alignment as 16-byte words.
//
// Word i of a row is the 16-byte aligned word of memory that holds entries
// [i*E - mis, i*E - mis + E), E = 16 / sizeof(T) and mis the row's offset within its
// first word.  Words that lie wholly inside the row move as one 16-byte access; the
// first and the last word of a row whose ends are not on 16 bytes move entry by entry,
// so nothing outside the row is read or written, whatever V and the row stride are.
#pragma once

#include "spec_device.cuh"

namespace spec {

inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }   // parts of a workspace

// Larger over the warp, NaN when any lane has it.
__device__ __forceinline__ float warp_max_nan(float x) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

template <typename T> struct NegInf;
template <> struct NegInf<float> { static constexpr uint32_t word = 0xff800000u; };
template <> struct NegInf<bf16_t> { static constexpr uint32_t word = 0xff80ff80u; };

// The words that are not whole, out of line: entries [e, e + E) of a row of V entries, -inf
// outside it, and the way back.
template <typename T>
__device__ __noinline__ uint4 edge_load(const T* p, int e, int V) {
    constexpr int E = 16 / (int)sizeof(T);
    uint32_t h[4] = {NegInf<T>::word, NegInf<T>::word, NegInf<T>::word, NegInf<T>::word};
#pragma unroll
    for (int k = 0; k < E; ++k) {
        if (e + k < 0 || e + k >= V) continue;
        if (sizeof(T) == 2) {
            const uint32_t v = reinterpret_cast<const unsigned short*>(p)[e + k];
            h[k >> 1] = (k & 1) ? (h[k >> 1] & 0xffffu) | (v << 16) : (h[k >> 1] & 0xffff0000u) | v;
        } else {
            h[k & 3] = reinterpret_cast<const uint32_t*>(p)[e + k];
        }
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}
template <typename T>
__device__ __noinline__ void edge_store(T* q, int e, int V, uint4 w) {
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 16 / (int)sizeof(T); ++k) {
        if (e + k < 0 || e + k >= V) continue;
        if (sizeof(T) == 2) reinterpret_cast<unsigned short*>(q)[e + k] = (unsigned short)(h[k >> 1] >> (16 * (k & 1)));
        else reinterpret_cast<uint32_t*>(q)[e + k] = h[k & 3];
    }
}

template <typename T>
struct RowWords {
    static constexpr int E = 16 / (int)sizeof(T);
    const T* p;
    int V;
    int mis;   // entries of the first word that lie before the row
    int n;     // words

    __device__ __forceinline__ RowWords(const T* row, int len)
        : p(row), V(len), mis((int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T))),
          n(len > 0 ? (int)(((long)mis + len + E - 1) / E) : 0) {}

    __device__ __forceinline__ int entry(int i) const { return i * E - mis; }
    __device__ __forceinline__ bool whole(int i) const {   // all but the first and the last are
        return (unsigned)(i - 1) < (unsigned)max(n - 2, 0) || (entry(i) >= 0 && entry(i) + E <= V);
    }
    // word i, entries outside the row as -inf
    __device__ __forceinline__ uint4 load(int i) const {
        if (!whole(i)) return edge_load<T>(p, entry(i), V);
        uint4 v;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p + entry(i)) : "memory");
        return v;
    }
    // word i into the row `q` of the same length and offset
    __device__ __forceinline__ void store(T* q, int i, const uint4& w) const {
        if (!whole(i)) return edge_store<T>(q, entry(i), V, w);
        asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};"
                     :: "l"(q + entry(i)), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
    }
};

// Entry k of a word as a float.
template <typename T>
__device__ __forceinline__ float word_entry(const uint4& w, int k) {
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
    if (sizeof(T) == 2) return __uint_as_float((k & 1) ? (h[k >> 1] & 0xffff0000u) : (h[k >> 1] << 16));
    return __uint_as_float(h[k & 3]);
}

// The same for a k known at run time only.
template <typename T>
__device__ __forceinline__ float word_pick(const uint4& w, int k) {
    const int r = sizeof(T) == 2 ? k >> 1 : k;
    const uint32_t h = (r & 2) ? ((r & 1) ? w.w : w.z) : ((r & 1) ? w.y : w.x);
    if (sizeof(T) == 2) return __uint_as_float((k & 1) ? (h & 0xffff0000u) : (h << 16));
    return __uint_as_float(h);
}

// Bits [e, e + 32) of a bit string, e >= 0 (one word past the end may be read).
__device__ __forceinline__ uint32_t bits_at(const uint32_t* w, int e) {
    return __funnelshift_r(w[e >> 5], w[(e >> 5) + 1], e & 31);
}

// The words of a row or of a segment of one.  ALIGNED: the segment starts on 16 bytes and is a whole
// number of words, as every segment does when rows are whole words apart and V is whole words.
// Without the tests for a row's ends the distillation loss of 448 rows of 248,320 bf16 takes
// 37.5 us instead of 44.3, the 64 largest of 256 rows 32.7 instead of 34.8.
template <typename T, bool ALIGNED>
struct SegWords {
    static constexpr int E = 16 / (int)sizeof(T);
    RowWords<T> r;
    __device__ __forceinline__ SegWords(const T* row, int len) : r(row, len) {}
    static bool fits(int ld, int V) { return ld % E == 0 && V % E == 0; }
    __device__ __forceinline__ int n() const { return ALIGNED ? r.V / E : r.n; }
    __device__ __forceinline__ int entry(int i) const { return ALIGNED ? i * E : r.entry(i); }
    __device__ __forceinline__ uint4 load(int i) const {
        if (!ALIGNED) return r.load(i);
        uint4 v;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(reinterpret_cast<const uint4*>(r.p) + i) : "memory");
        return v;
    }
    __device__ __forceinline__ void store(T* q, int i, const uint4& w) const {
        if (!ALIGNED) return r.store(q, i, w);
        asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};"
                     :: "l"(reinterpret_cast<uint4*>(q) + i), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
    }
    // the bits of a mask that go with word i, as loaded, and then bit k for entry k; `left` words
    // of mask from the segment's first
    __device__ __forceinline__ uint32_t mask_word(const uint32_t* mask, int left, int i) const {
        if (ALIGNED) return (uint32_t)__ldg(reinterpret_cast<const uint8_t*>(mask) + (E == 8 ? i : i >> 1));
        const int e = entry(i), e0 = max(e, 0), at = e0 & 31;
        const uint32_t lo = __ldg(mask + (e0 >> 5));
        const uint32_t hi = at + E > 32 && (e0 >> 5) + 1 < left ? __ldg(mask + (e0 >> 5) + 1) : 0u;
        return (__funnelshift_r(lo, hi, at) << (e0 - e)) & ((1u << E) - 1u);
    }
    __device__ __forceinline__ uint32_t allowed(uint32_t loaded, int i) const {
        return ALIGNED && E == 4 ? (loaded >> (4 * (i & 1))) & 15u : loaded;
    }
    // the entries of word i in the segment's array, which has E entries of room before it and
    // as many behind it
    __device__ __forceinline__ void floats(const float* a, int i, float (&o)[E]) const {
#pragma unroll
        for (int k = 0; k < E; k += 4) {
            if (ALIGNED) {
                const float4 v = *reinterpret_cast<const float4*>(a + i * E + k);
                o[k] = v.x; o[k + 1] = v.y; o[k + 2] = v.z; o[k + 3] = v.w;
            } else {
#pragma unroll
                for (int h = k; h < k + 4; ++h) o[h] = a[entry(i) + h];
            }
        }
    }
    // the bits of word i in the segment's bit string, which has a clear word before it and
    // behind it
    __device__ __forceinline__ uint32_t bits(const uint32_t* bits, int i) const {
        if (ALIGNED) {
            const uint8_t* m = reinterpret_cast<const uint8_t*>(bits);
            return E == 8 ? (uint32_t)m[i] : ((uint32_t)m[i >> 1] >> (4 * (i & 1))) & 15u;
        }
        return bits_at(bits - 1, entry(i) + 32) & ((1u << E) - 1u);
    }
};

// Weights relative to a reference m, in base 2: entry x of a row weighs 2^((x - m) c), c = log2(e) / t,
// and sums that belong to different references are brought together by the same expression
// (ref_rel).  The streaming loops form 2^(x c - R(m)) instead, with R(m) = m c rounded once and x c
// exact inside an FFMA; what the rounding has moved all of a sum's weights by, 2^4 at most while
// |m c| <= kRefNear, is taken back once per sum (ref_fix).  Beyond (rows masked with -1e10, -1e30 or
// the type's lowest value, large logits over a small temperature) it would leave float32's range,
// and m c itself can overflow: there the loops take the difference first as well, out of line.
constexpr float kRefNear = 67108864.0f;   // 2^26
__device__ __forceinline__ bool ref_near(float y) { return fabsf(y) <= kRefNear; }
__device__ __forceinline__ float ref_rel(float x, float m, float c) { return (x - m) * c; }   // log2 weight of x, m > -inf
__device__ __forceinline__ float ref_fix(float m, float c) {   // takes words_sum's R(m) to m
    const float y = m * c;
    return ref_near(y) ? ex2(-fmaf(m, c, -y)) : 1.0f;
}
// ln of a sum relative to m
__device__ __forceinline__ float ref_log(float m, float s, float inv_t) { return fmaf(m, inv_t, logf(s)); }
// log2 of what a sum of words_sum's relative to a is worth relative to b >= a > -inf
static __device__ __noinline__ float ref_step_far(float a, float b, float c) {
    const float x = a * c, y = b * c;
    if (ref_near(y)) return fmaf(a, c, -y);
    return ref_near(x) ? -fmaf(b, c, -x) : (a - b) * c;
}
__device__ __forceinline__ float ref_step(float a, float b, float c) {
    const float x = a * c, y = b * c;
    return ref_near(x) && ref_near(y) ? x - y : ref_step_far(a, b, c);
}
// A word's weights relative to a reference beyond kRefNear: out of line, since hardly any row has
// one and the streaming loops are short without it.
template <typename T>
__device__ __noinline__ float word_sum_far(uint4 w, float m, float c) {
    float s = 0.0f;
    for (int k = 0; k < 16 / (int)sizeof(T); ++k) s += ex2((word_pick<T>(w, k) - m) * c);
    return s;
}
// The sum of the weights of N words relative to m, R(m) within kRefNear (0 for m = -inf).
template <typename T, int N>
__device__ __forceinline__ float words_sum(const uint4 (&w)[N], float m, float c) {
    const float x = m * c;
    f2x acc[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
    const f2x cc = f2_pack(c, c);
    if (ref_near(x)) {
        const f2x mm = f2_pack(-x, -x);
#pragma unroll
        for (int h = 0; h < N; ++h)
#pragma unroll
            for (int k = 0; k < 16 / (int)sizeof(T); k += 2)
                acc[(k >> 1) & 1] = f2_add(acc[(k >> 1) & 1],
                    f2_ex2(f2_fma(f2_pack(word_entry<T>(w[h], k), word_entry<T>(w[h], k + 1)), cc, mm)));
    } else {
        if (!(m > -INFINITY)) return 0.0f;
        float s = 0.0f;
        for (int h = 0; h < N; ++h) s += word_sum_far<T>(w[h], m, c);
        return s;
    }
    const float2 a = f2_unpack(acc[0]), b = f2_unpack(acc[1]);
    return (a.x + a.y) + (b.x + b.y);
}

// -inf in the entries of a word whose bit is set.
template <typename T>
__device__ __forceinline__ uint4 word_without(const uint4& w, uint32_t bits) {
    uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 16 / (int)sizeof(T); ++k) {
        if (!((bits >> k) & 1u)) continue;
        if (sizeof(T) == 2) h[k >> 1] = (k & 1) ? (h[k >> 1] & 0xffffu) | 0xff800000u : (h[k >> 1] & 0xffff0000u) | 0xff80u;
        else h[k & 3] = 0xff800000u;
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// E floats rounded (to nearest even for bf16) into a word.
template <typename T>
__device__ __forceinline__ uint4 word_of(const float (&x)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[k]) : "f"(x[2 * k + 1]), "f"(x[2 * k]));
        return make_uint4(h[0], h[1], h[2], h[3]);
    } else {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
}

}  // namespace spec
