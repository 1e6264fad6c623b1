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

template <typename T> struct NegInf;
template <> struct NegInf<float> { static constexpr uint32_t word = 0xff800000u; };
template <> struct NegInf<bf16_t> { static constexpr uint32_t word = 0xff80ff80u; };

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
    __device__ __forceinline__ bool whole(int i) const { return entry(i) >= 0 && entry(i) + E <= V; }

    __device__ __forceinline__ uint32_t raw(int e) const {   // entry e's bits, -inf outside the row
        if (e < 0 || e >= V) return NegInf<T>::word & (sizeof(T) == 2 ? 0xffffu : 0xffffffffu);
        if (sizeof(T) == 2) return reinterpret_cast<const unsigned short*>(p)[e];
        return reinterpret_cast<const uint32_t*>(p)[e];
    }
    // word i, entries outside the row as -inf
    __device__ __forceinline__ uint4 load(int i) const {
        if (whole(i)) {
            uint4 v;
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p + entry(i)) : "memory");
            return v;
        }
        const int e = entry(i);
        if (sizeof(T) == 2)
            return make_uint4(raw(e) | (raw(e + 1) << 16), raw(e + 2) | (raw(e + 3) << 16),
                              raw(e + 4) | (raw(e + 5) << 16), raw(e + 6) | (raw(e + 7) << 16));
        return make_uint4(raw(e), raw(e + 1), raw(e + 2), raw(e + 3));
    }
    // word i into the row `q` of the same length and offset
    __device__ __forceinline__ void store(T* q, int i, const uint4& w) const {
        const int e = entry(i);
        if (whole(i)) {
            asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};"
                         :: "l"(q + e), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
            return;
        }
        const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < E; ++k) {
            if (e + k < 0 || e + k >= V) continue;
            if (sizeof(T) == 2)
                reinterpret_cast<unsigned short*>(q)[e + k] = (unsigned short)(h[k >> 1] >> (16 * (k & 1)));
            else
                reinterpret_cast<uint32_t*>(q)[e + k] = h[k & 3];
        }
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
