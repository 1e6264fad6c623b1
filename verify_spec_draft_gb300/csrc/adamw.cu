// adamw.cu - one AdamW step over many tensors (spec_adamw).
//
// Every entry is independent but for the scale that 128 entries of an 8-bit state share, so
// a step is one pass: read p, g, m, v, write p, m, v.  A warp takes blocks of 128 entries, a
// lane 4 neighbours of each, so every access is whole sectors and a block's largest magnitude is
// one warp reduction.  The tensors' table lies in the kernel's parameters: nothing is copied to
// the device, and a captured step replays as it is.
// Bound by memory: 28 bytes an entry with a bf16 parameter and gradient, a master and 32-bit states (127 M entries
// 567 to 578 us, 92 to 94 % of the measured copy rate), 16 with 8-bit ones (371 us, 83 %: the codes' rounding
// takes the issue slots 66 % of the time).  Tensors that do not lie on whole words, and those of less than a chunk, go
// entry by entry (adam_edge): 16 M entries, bf16 with masters, take 85 us on words and 164 off them, 68 and 145 with
// 8-bit states.
#include "internal.h"
#include "spec_device.cuh"

#include <cuda_fp16.h>
#include <string.h>
#include <type_traits>

namespace spec {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamUnroll = 2;                                   // blocks of a warp in flight
constexpr int kAdamBlock = SPEC_ADAMW_BLOCK;
constexpr int kAdamUnit = kAdamUnroll * kAdamBlock;              // entries of a warp's turn
constexpr int kAdamChunk = kAdamWarps * kAdamUnit;               // entries of a CTA's turn
constexpr int kAdamSpan = 16;                                    // most chunks in a row that a CTA takes
constexpr int kAdamCtas = 4;                                     // per SM
static_assert(kAdamBlock == 128, "a lane takes 4 entries of a block");

enum { kAdamHalf = 1, kAdamGradHalf = 2, kAdamPacked = 4, kAdamVec = 8 };

struct AdamwTensor {
    float* p;               // the float32 parameter, or the master of a bf16 one
    bf16_t* half;           // the bf16 parameter
    const void* grad;
    void *m, *v;
    float *m_scale, *v_scale;
    long n;
    unsigned first;         // chunks before this tensor
    unsigned kind;
};
template <int CAP>
struct AdamwArgs {
    AdamwTensor t[CAP];
    int n, base;            // tensors of this launch, and the first one's index
    unsigned chunks, span;
    int advance;            // the call's last launch: step goes up
    int32_t* step;
    const float* grad_scale;
    double beta1, beta2;
    float lr, keep, eps;                // keep = 1 - lr weight_decay
    float b1, b1c, b2, b2c;             // beta, 1 - beta
    uint32_t key[20];                   // Philox' round keys
    unsigned* status;
    unsigned* done;
};

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC'11, table 2); the round keys are the launch's.
__device__ __forceinline__ uint4 philox4x32(const uint32_t* key, uint64_t block, uint32_t c2, uint32_t c3) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ key[2 * r];
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ key[2 * r + 1];
        c3 = (uint32_t)a;
    }
    return make_uint4(c0, c1, c2, c3);
}

// 4 entries as two pairs.
struct Quad {
    f2x a, b;
    __device__ __forceinline__ Quad() {}
    __device__ __forceinline__ Quad(f2x x, f2x y) : a(x), b(y) {}
    __device__ __forceinline__ explicit Quad(float x) : a(f2_pack(x, x)), b(f2_pack(x, x)) {}
    __device__ __forceinline__ Quad(float x, float y, float z, float w) : a(f2_pack(x, y)), b(f2_pack(z, w)) {}
    __device__ __forceinline__ float4 get() const {
        const float2 x = f2_unpack(a), y = f2_unpack(b);
        return make_float4(x.x, x.y, y.x, y.y);
    }
};
__device__ __forceinline__ Quad operator*(const Quad& x, const Quad& y) { return Quad(f2_mul(x.a, y.a), f2_mul(x.b, y.b)); }
// (by fours: a product of pairs and a sum of pairs are fused, whatever their rounding is given as)
__device__ __forceinline__ Quad operator+(const Quad& x, const Quad& y) {
    const float4 a = x.get(), b = y.get();
    return Quad(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}
__device__ __forceinline__ Quad quad_fma(const Quad& x, const Quad& y, const Quad& z) {
    return Quad(f2_fma(x.a, y.a, z.a), f2_fma(x.b, y.b, z.b));
}

// e4m3 codes' values.
__device__ __forceinline__ Quad e4m3_values(uint32_t codes) {
    uint32_t lo, hi;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return Quad(x.x, x.y, y.x, y.y);
}
// The code of |y| < 256 in the top byte, up with probability (what is left) / (the code's spacing): 16
// random bits (at bits 8-23) are added to the bits below, and the carry goes up.  A float's exponent
// and mantissa, less the difference of the biases, are the code and 20 bits; below 2^-6, where
// the spacing stays 2^-9, those of |y| + 2^-6 less its own code are.  Each is the larger where it holds.
__device__ __forceinline__ uint32_t e4m3_random(float y, uint32_t random) {
    const int n = (int)((__float_as_uint(y) & 0x7fffffffu) - (960u << 20));
    const int d = (int)(__float_as_uint(__fadd_rz(fabsf(y), 0x1p-6f)) - (968u << 20));
    return ((uint32_t)max(n, d) << 4) + random;
}
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

struct AdamwHyper {
    float b1, b1c, b2, b2c, keep, eps, size, root, clip;
    const uint32_t* key;
    uint32_t T;
};

// 4 entries: m and v (PACKED: v is its root) and the parameter replaced.  Products and sums that a
// state comes from are rounded one by one, in the order of the formulas, so that a code does not
// depend on what a compiler fuses.  What the parameter alone sees (the root's and the quotient's
// last bits, 2^-22 of a step) is not.
template <bool PACKED>
__device__ __forceinline__ bool adam_quad(const AdamwHyper& h, Quad& p, Quad g, Quad& m, Quad& v) {
    g = g * Quad(h.clip);
    const Quad m1 = m * Quad(h.b1) + g * Quad(h.b1c);
    const Quad v1 = (PACKED ? v * v : v) * Quad(h.b2) + g * Quad(h.b2c) * g;
    const float4 w = v1.get();
    float r[4] = {w.x, w.y, w.z, w.w}, q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (PACKED) r[k] = __fsqrt_rn(r[k]);
        else asm("sqrt.approx.f32 %0, %1;" : "=f"(r[k]) : "f"(r[k]));
    }
    const Quad root(r[0], r[1], r[2], r[3]);
    const float4 den = quad_fma(root, Quad(h.root), Quad(h.eps)).get();
    const float e[4] = {den.x, den.y, den.z, den.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q[k]) : "f"(e[k]));
    const Quad p1 = quad_fma(m1 * Quad(q[0], q[1], q[2], q[3]), Quad(-h.size), p * Quad(h.keep));
    // 0 unless a gradient is not finite, or too large
    const float4 x = quad_fma(m1, Quad(0.0f), v1 * Quad(0.0f)).get();
    const bool fine = (x.x + x.y) + (x.z + x.w) == 0.0f;
    if (fine) {
        p = p1;
        m = m1;
        v = PACKED ? root : v1;
    } else {   // those entries stay
        const float4 a = p.get(), b = m.get(), c = v.get(), a1 = p1.get(), b1 = m1.get(), c1 = (PACKED ? root : v1).get();
        p = Quad(x.x == 0.0f ? a1.x : a.x, x.y == 0.0f ? a1.y : a.y, x.z == 0.0f ? a1.z : a.z, x.w == 0.0f ? a1.w : a.w);
        m = Quad(x.x == 0.0f ? b1.x : b.x, x.y == 0.0f ? b1.y : b.y, x.z == 0.0f ? b1.z : b.z, x.w == 0.0f ? b1.w : b.w);
        v = Quad(x.x == 0.0f ? c1.x : c.x, x.y == 0.0f ? c1.y : c.y, x.z == 0.0f ? c1.z : c.z, x.w == 0.0f ? c1.w : c.w);
    }
    return !fine;
}

// 4 entries of a block in 8 bits, their sign beside 7 bits (ROOT: none, and 0 only for 0: a root above 0
// is 2^-75 at least, whose bits are above 2^24).  m takes the low half of a random word, v the high one.
template <bool ROOT>
__device__ __forceinline__ uint32_t pack4(const Quad& v, const uint4& random, float& scale) {
    const float4 x = v.get();
    const float top = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
    const uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    const uint32_t e = (uint32_t)max((int)(u >> 23) - 7, 1);
    scale = __uint_as_float(e << 23);
    const float4 y4 = (v * Quad(__uint_as_float((254u - e) << 23))).get();
    const float y[4] = {y4.x, y4.y, y4.z, y4.w}, z[4] = {x.x, x.y, x.z, x.w};
    const uint32_t rnd[4] = {random.x, random.y, random.z, random.w};
    uint32_t code[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        code[k] = e4m3_random(y[k], __byte_perm(rnd[k], 0u, ROOT ? 0x4324 : 0x4104));
        if (ROOT) code[k] = max(code[k], min(__float_as_uint(z[k]), 1u << 24));
    }
    uint32_t w = top_bytes(code[0], code[1], code[2], code[3]);
    if (!ROOT)
        w |= top_bytes(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3])) & 0x80808080u;
    return w;
}

template <typename T> __device__ __forceinline__ Quad load4(const T* a) {
    if constexpr (sizeof(T) == 4) {
        const float4 w = __ldcs(reinterpret_cast<const float4*>(a));
        return Quad(w.x, w.y, w.z, w.w);
    } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(a));
        return Quad(bf2_widen(w.x), bf2_widen(w.y));
    }
}
__device__ __forceinline__ uint2 half4(const float4& x) {
    return make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// A warp's turn of whole blocks, every access a word of 4 entries.  Lane l holds the scales of the l-th
// block from a line of 32 on; `block` is the turn's first one's place in it.  (Addresses are formed anew
// at every turn: kept in registers, eight pointers spill.)
template <bool HALF, bool GRAD16, bool PACKED>
__device__ __forceinline__ bool adam_blocks(const AdamwTensor& t, const AdamwHyper& h, int index, long at, int lane,
                                            int block, float& m_scale, float& v_scale) {
    typedef typename std::conditional<GRAD16, bf16_t, float>::type G;
    Quad p[kAdamUnroll], g[kAdamUnroll], m[kAdamUnroll], v[kAdamUnroll];
    uint32_t cm[kAdamUnroll], cv[kAdamUnroll];
    bool bad = false;
    const long first = at + lane * 4;
    float* tp = t.p + first;
    const G* tg = reinterpret_cast<const G*>(t.grad) + first;
    uint8_t *m8 = reinterpret_cast<uint8_t*>(t.m) + first, *v8 = reinterpret_cast<uint8_t*>(t.v) + first;
    float *m32 = reinterpret_cast<float*>(t.m) + first, *v32 = reinterpret_cast<float*>(t.v) + first;
#pragma unroll
    for (int q = 0; q < kAdamUnroll; ++q) {
        p[q] = load4(tp + q * kAdamBlock);
        g[q] = load4(tg + q * kAdamBlock);
        if (PACKED) {
            cm[q] = __ldcs(reinterpret_cast<const uint32_t*>(m8 + q * kAdamBlock));
            cv[q] = __ldcs(reinterpret_cast<const uint32_t*>(v8 + q * kAdamBlock));
        } else {
            m[q] = load4(m32 + q * kAdamBlock);
            v[q] = load4(v32 + q * kAdamBlock);
        }
    }
#pragma unroll
    for (int q = 0; q < kAdamUnroll; ++q) {
        if (PACKED) {
            m[q] = e4m3_values(cm[q]) * Quad(__shfl_sync(0xffffffffu, m_scale, block + q));
            v[q] = e4m3_values(cv[q]) * Quad(__shfl_sync(0xffffffffu, v_scale, block + q));
        }
        bad |= adam_quad<PACKED>(h, p[q], g[q], m[q], v[q]);
        const float4 x = p[q].get();
        __stcs(reinterpret_cast<float4*>(tp + q * kAdamBlock), x);
        if (HALF) __stcs(reinterpret_cast<uint2*>(t.half + first + q * kAdamBlock), half4(x));
        if (PACKED) {
            const uint4 w = philox4x32(h.key, (uint64_t)(first + q * kAdamBlock) / 4, h.T, (uint32_t)index);
            float a, b;
            __stcs(reinterpret_cast<uint32_t*>(m8 + q * kAdamBlock), pack4<false>(m[q], w, a));
            __stcs(reinterpret_cast<uint32_t*>(v8 + q * kAdamBlock), pack4<true>(v[q], w, b));
            m_scale = lane == block + q ? a : m_scale;
            v_scale = lane == block + q ? b : v_scale;
        } else {
            __stcs(reinterpret_cast<float4*>(m32 + q * kAdamBlock), m[q].get());
            __stcs(reinterpret_cast<float4*>(v32 + q * kAdamBlock), v[q].get());
        }
    }
    return bad;
}

// A warp's turns from entry `at` on: `turns` of them, 32 blocks at a time, whose scales are a line.
template <bool HALF, bool GRAD16, bool PACKED>
__device__ __forceinline__ bool adam_turns(const AdamwTensor& t, const AdamwHyper& h, int index, long at, int turns, int lane) {
    bool bad = false;
    while (turns > 0) {
        const int now = min(turns, 32 / kAdamUnroll);
        const bool mine = PACKED && lane < now * kAdamUnroll;
        const long b = at / kAdamBlock + lane;
        float ms = mine ? t.m_scale[b] : 0.0f, vs = mine ? t.v_scale[b] : 0.0f;
#pragma unroll 1
        for (int q = 0; q < now; ++q, at += kAdamUnit)
            bad |= adam_blocks<HALF, GRAD16, PACKED>(t, h, index, at, lane, q * kAdamUnroll, ms, vs);
        if (mine) {
            t.m_scale[b] = ms;
            t.v_scale[b] = vs;
        }
        turns -= now;
    }
    return bad;
}

// A block entry by entry: a tensor's end, or one that does not lie on whole words.
static __device__ __noinline__ bool adam_edge(const AdamwTensor& t, const AdamwHyper& h, int index, long at, int lane) {
    float p[4], g[4], m[4], v[4];
    const long first = at + lane * 4;
    const int n = (int)max(0l, min(4l, t.n - first));
    const bool packed = t.kind & kAdamPacked;
    uint8_t *m8 = reinterpret_cast<uint8_t*>(t.m) + first, *v8 = reinterpret_cast<uint8_t*>(t.v) + first;
    float *m32 = reinterpret_cast<float*>(t.m) + first, *v32 = reinterpret_cast<float*>(t.v) + first;
    uint32_t cm = 0u, cv = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {   // (what is beyond the end is all 0, and stays)
        p[k] = g[k] = m[k] = v[k] = 0.0f;
        if (k >= n) continue;
        p[k] = t.p[first + k];
        g[k] = t.kind & kAdamGradHalf ? to_float(reinterpret_cast<const bf16_t*>(t.grad)[first + k])
                                      : reinterpret_cast<const float*>(t.grad)[first + k];
        if (packed) {
            cm |= (uint32_t)m8[k] << (8 * k);
            cv |= (uint32_t)v8[k] << (8 * k);
        } else {
            m[k] = m32[k];
            v[k] = v32[k];
        }
    }
    Quad pq(p[0], p[1], p[2], p[3]), mq(m[0], m[1], m[2], m[3]), vq(v[0], v[1], v[2], v[3]);
    const Quad gq(g[0], g[1], g[2], g[3]);
    bool bad;
    if (packed) {
        mq = e4m3_values(cm) * Quad(t.m_scale[at / kAdamBlock]);
        vq = e4m3_values(cv) * Quad(t.v_scale[at / kAdamBlock]);
        bad = adam_quad<true>(h, pq, gq, mq, vq);
        const uint4 w = philox4x32(h.key, (uint64_t)first / 4, h.T, (uint32_t)index);
        float a, b;
        cm = pack4<false>(mq, w, a);
        cv = pack4<true>(vq, w, b);
        __syncwarp();   // every lane has read the scales
        if (lane == 0) {
            t.m_scale[at / kAdamBlock] = a;
            t.v_scale[at / kAdamBlock] = b;
        }
    } else {
        bad = adam_quad<false>(h, pq, gq, mq, vq);
    }
    const float4 x = pq.get(), y = mq.get(), z = vq.get();
    const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w};
    const uint2 hw = half4(x);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k >= n) continue;
        t.p[first + k] = xs[k];
        if (t.kind & kAdamHalf) t.half[first + k] = (bf16_t)((k < 2 ? hw.x : hw.y) >> (16 * (k & 1)));
        if (packed) {
            m8[k] = (uint8_t)(cm >> (8 * k));
            v8[k] = (uint8_t)(cv >> (8 * k));
        } else {
            m32[k] = ys[k];
            v32[k] = zs[k];
        }
    }
    return bad;
}

template <int CAP>
__global__ void __launch_bounds__(kAdamThreads, kAdamCtas) adamw_kernel(const __grid_constant__ AdamwArgs<CAP> a) {
    __shared__ float s_size, s_root;
    __shared__ int s_step;
    if (threadIdx.x == 0) {
        const int step = *a.step;
        s_step = step;
        // beta^T by squares
        double p1 = 1.0, p2 = 1.0, q1 = a.beta1, q2 = a.beta2;
        for (uint32_t e = (uint32_t)step + 1u; e; e >>= 1) {
            if (e & 1u) { p1 *= q1; p2 *= q2; }
            q1 *= q1;
            q2 *= q2;
        }
        s_size = a.lr / (float)(1.0 - p1);
        s_root = 1.0f / sqrtf((float)(1.0 - p2));
    }
    __syncthreads();
    const int step = s_step, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool fine = step >= 0 && step < 0x7fffffff;
    AdamwHyper h;
    h.b1 = a.b1; h.b1c = a.b1c; h.b2 = a.b2; h.b2c = a.b2c;
    h.keep = a.keep; h.eps = a.eps; h.size = s_size; h.root = s_root;
    h.clip = a.grad_scale ? *a.grad_scale : 1.0f;
    h.key = a.key; h.T = (uint32_t)step + 1u;
    bool bad = false;
    int at_tensor = 0;
    // a.span chunks in a row at a time: what is looked up per tensor is spread over them
    for (unsigned long long c0 = (unsigned long long)blockIdx.x * a.span; fine && c0 < a.chunks; c0 += (unsigned long long)gridDim.x * a.span) {
        unsigned c = (unsigned)c0;
        const unsigned end = (unsigned)min((unsigned long long)a.chunks, c0 + a.span);
        while (c < end) {
            // the one that chunk c is of (2000 tensors of 1000 entries, 400 a launch: 66 us, looked for one by one 204)
            for (int behind = a.n; at_tensor + 1 < behind && a.t[at_tensor + 1].first <= c;) {
                const int mid = (at_tensor + 1 + behind) / 2;
                if (a.t[mid].first <= c) at_tensor = mid;
                else behind = mid;
            }
            const AdamwTensor& t = a.t[at_tensor];
            const int index = a.base + at_tensor;
            const unsigned kind = t.kind;
            const long start = (long)(c - t.first) * kAdamChunk, left = t.n - start;
            const int whole = kind & kAdamVec ? (int)min((long)(end - c), left / kAdamChunk) : 0;
            if (whole == 0) {   // a tensor's end, or any part of one that is not aligned: its blocks over the warps
                const long stop = min(t.n, start + kAdamChunk);
                for (long e = start + warp * kAdamBlock; e < stop; e += kAdamWarps * kAdamBlock)
                    bad |= adam_edge(t, h, index, e, lane);
                ++c;
                continue;
            }
            c += (unsigned)whole;
            // a warp's entries lie in a row (a scale's sector, written by one warp in time: 394 us when this was chosen; by several: 480)
            const long at = start + (long)warp * whole * kAdamUnit;
            switch (kind & 7u) {
#define SPEC_ADAM_CASE(K)                                                                                             \
    case K:                                                                                                           \
        bad |= adam_turns<((K) & kAdamHalf) != 0, ((K) & kAdamGradHalf) != 0, ((K) & kAdamPacked) != 0>(t, h, index,  \
                                                                                                      at, whole, lane); \
        break;
                SPEC_ADAM_CASE(0) SPEC_ADAM_CASE(1) SPEC_ADAM_CASE(2) SPEC_ADAM_CASE(3)
                SPEC_ADAM_CASE(4) SPEC_ADAM_CASE(5) SPEC_ADAM_CASE(6) SPEC_ADAM_CASE(7)
#undef SPEC_ADAM_CASE
            }
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, SPEC_DEV_NONFINITE);
    if (!a.advance) return;
    if (last_block_done(a.done, gridDim.x) && threadIdx.x == 0) {   // every CTA has read the step
        *a.done = 0u;
        if (fine) *a.step = step + 1;
        else atomicOr(a.status, SPEC_DEV_TOKEN);
    }
}

template <int CAP>
static cudaError_t adamw_typed(const AdamwCall& c, cudaStream_t stream) {
    AdamwArgs<CAP> a;
    memset(&a, 0, sizeof(a));
    a.step = c.step;
    a.grad_scale = c.grad_scale;
    a.beta1 = c.beta1;
    a.beta2 = c.beta2;
    a.lr = (float)c.lr;
    a.keep = (float)(1.0 - c.lr * c.weight_decay);
    a.eps = (float)c.eps;
    a.b1 = (float)c.beta1;
    a.b1c = (float)(1.0 - c.beta1);
    a.b2 = (float)c.beta2;
    a.b2c = (float)(1.0 - c.beta2);
    for (uint32_t r = 0; r < 10; ++r) {
        a.key[2 * r] = (uint32_t)c.seed + r * 0x9E3779B9u;
        a.key[2 * r + 1] = (uint32_t)(c.seed >> 32) + r * 0xBB67AE85u;
    }
    a.status = &reinterpret_cast<WsHeader*>(c.ws)->status;
    a.done = &reinterpret_cast<WsHeader*>(c.ws)->done[0];
    const unsigned most = (unsigned)(device_sm_count() * kAdamCtas);
    int i = 0;
    do {
        a.base = i;
        a.n = 0;
        uint64_t chunks = 0;
        for (; i < c.n_tensors && a.n < CAP; ++i) {
            const spec_adamw_tensor& s = c.tensors[i];
            const uint64_t mine = ((uint64_t)s.n + kAdamChunk - 1) / kAdamChunk;
            if (chunks + mine > 0xffffff00ull) break;
            AdamwTensor& t = a.t[a.n++];
            const bool half = s.param_dtype == SPEC_BF16, packed = s.state_bits == 8;
            t.p = half ? s.master : reinterpret_cast<float*>(s.param);
            t.half = half ? reinterpret_cast<bf16_t*>(s.param) : nullptr;
            t.grad = s.grad;
            t.m = s.m;
            t.v = s.v;
            t.m_scale = s.m_scale;
            t.v_scale = s.v_scale;
            t.n = s.n;
            t.first = (unsigned)chunks;
            auto on = [](const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; };
            const bool vec = on(t.p, 16) && on(t.half, 8) && on(t.grad, s.grad_dtype == SPEC_BF16 ? 8 : 16) &&
                             on(t.m, packed ? 4 : 16) && on(t.v, packed ? 4 : 16);
            t.kind = (half ? kAdamHalf : 0) | (s.grad_dtype == SPEC_BF16 ? kAdamGradHalf : 0) |
                     (packed ? kAdamPacked : 0) | (vec ? kAdamVec : 0);
            chunks += mine;
        }
        a.chunks = (unsigned)chunks;
        a.advance = i >= c.n_tensors;
        // enough spans that the CTAs end within a few per cent of one another
        const unsigned span = a.chunks / (most * 8u);
        a.span = span < 1u ? 1u : (span < (unsigned)kAdamSpan ? span : (unsigned)kAdamSpan);
        const unsigned spans = (a.chunks + a.span - 1) / a.span;
        const unsigned grid = spans < most ? (spans ? spans : 1u) : most;
        adamw_kernel<CAP><<<grid, kAdamThreads, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    } while (i < c.n_tensors);
    return cudaSuccess;
}

// The table travels with each launch: a short one for a few tensors, the largest that the
// parameters take for many.
cudaError_t adamw_launch(const AdamwCall& c, cudaStream_t stream) {
    return c.n_tensors <= 32 ? adamw_typed<32>(c, stream) : adamw_typed<400>(c, stream);
}

}  // namespace spec
