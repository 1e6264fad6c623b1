// adamw.cu - one AdamW step over many tensors (spec_adamw).
//
// Every entry is independent but for the scale that 128 entries of an 8-bit state share, so
// a step is one pass: read p, g, m, v, write p, m, v.  A warp takes blocks of 128 entries, a
// lane 4 neighbours of each, so every access is whole sectors and a block's largest magnitude is
// one warp reduction.  The tensors' table lies in the kernel's parameters: nothing is copied to
// the device, and a captured step replays as it is.
#include "internal.h"
#include "spec_device.cuh"

#include <string.h>
#include <type_traits>

namespace spec {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamUnroll = 2;                                   // blocks of a warp in flight
constexpr int kAdamBlock = SPEC_ADAMW_BLOCK;
constexpr int kAdamChunk = kAdamWarps * kAdamUnroll * kAdamBlock;   // entries of a CTA's turn
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
    unsigned chunks;
    int advance;            // the call's last launch: step goes up
    int32_t* step;
    const float* grad_scale;
    double beta1, beta2;
    float lr, keep, eps;                // keep = 1 - lr weight_decay
    float b1, b1c, b2, b2c;             // beta, 1 - beta
    uint32_t k0, k1;
    unsigned* status;
    unsigned* done;
};

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC'11, table 2)
__device__ __forceinline__ uint4 philox4x32(uint32_t k0, uint32_t k1, uint64_t block, uint32_t c2, uint32_t c3) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// An e4m3 code's value (exact: its exponent and mantissa in a float's, then the bias).
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    return __uint_as_float((code & 0x7fu) << 20 | (code & 0x80u) << 24) * 0x1p120f;
}
// The code of |y| < 256, up with probability (what is left) / (the code's spacing), by 16
// random bits added to the bits that go: below 2^-6 those of a fixed-point number, above it
// the mantissa's, whose carry goes into the exponent.
__device__ __forceinline__ uint32_t e4m3_random(float y, uint32_t random) {
    const uint32_t u = __float_as_uint(y) & 0x7fffffffu;
    const uint32_t normal = ((u + (random << 4)) >> 20) - 960u;
    const uint32_t small = ((uint32_t)(__uint_as_float(u) * 0x1p25f) + random) >> 16;
    return u >= 0x3c800000u ? normal : small;
}

struct AdamwHyper {
    float b1, b1c, b2, b2c, keep, eps, size, root, clip;
    uint32_t k0, k1, T;
};

// One entry: m and v (`packed`: v is its root) replaced, the new parameter returned.  Products and
// sums are rounded one by one, in the order of the formulas, so that a state held in 8 bits is
// the same whatever a compiler fuses: a code must not depend on that.
template <bool PACKED>
__device__ __forceinline__ float adam_entry(const AdamwHyper& h, float p, float g, float& m, float& v, bool& bad) {
    g = __fmul_rn(g, h.clip);
    const float v0 = PACKED ? __fmul_rn(v, v) : v;
    const float m1 = __fadd_rn(__fmul_rn(m, h.b1), __fmul_rn(g, h.b1c));
    const float v1 = __fadd_rn(__fmul_rn(v0, h.b2), __fmul_rn(__fmul_rn(g, h.b2c), g));
    if (!(fabsf(m1) < INFINITY && v1 < INFINITY)) {   // g is not finite, or too large
        bad = true;
        return p;
    }
    const float r = PACKED ? __fsqrt_rn(v1) : sqrtf(v1);
    m = m1;
    v = PACKED ? r : v1;
    return p * h.keep - h.size * __fdividef(m1, fmaf(r, h.root, h.eps));
}

// 4 neighbouring entries of an array, n of them in it (VEC: whole words where all are)
template <bool VEC, typename T>
__device__ __forceinline__ void load4(const T* a, int n, float (&o)[4]) {
    if (VEC && n == 4) {
        if constexpr (sizeof(T) == 4) {
            const float4 w = __ldcs(reinterpret_cast<const float4*>(a));
            o[0] = w.x; o[1] = w.y; o[2] = w.z; o[3] = w.w;
        } else {
            const uint2 w = __ldcs(reinterpret_cast<const uint2*>(a));
            o[0] = __uint_as_float(w.x << 16); o[1] = __uint_as_float(w.x & 0xffff0000u);
            o[2] = __uint_as_float(w.y << 16); o[3] = __uint_as_float(w.y & 0xffff0000u);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = k < n ? to_float(a[k]) : 0.0f;
}
template <bool VEC>
__device__ __forceinline__ uint32_t load4_codes(const uint8_t* a, int n) {
    if (VEC && n == 4) return __ldcs(reinterpret_cast<const uint32_t*>(a));
    uint32_t w = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < n) w |= (uint32_t)a[k] << (8 * k);
    return w;
}
template <bool VEC>
__device__ __forceinline__ void store4(float* a, int n, const float (&x)[4]) {
    if (VEC && n == 4) {
        __stcs(reinterpret_cast<float4*>(a), make_float4(x[0], x[1], x[2], x[3]));
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < n) a[k] = x[k];
}
template <bool VEC>
__device__ __forceinline__ void store4_half(bf16_t* a, int n, const float (&x)[4]) {
    uint32_t lo, hi;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x[3]), "f"(x[2]));
    if (VEC && n == 4) {
        __stcs(reinterpret_cast<uint2*>(a), make_uint2(lo, hi));
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < n) a[k] = (bf16_t)((k < 2 ? lo : hi) >> (16 * (k & 1)));
}
template <bool VEC>
__device__ __forceinline__ void store4_codes(uint8_t* a, int n, uint32_t w) {
    if (VEC && n == 4) {
        __stcs(reinterpret_cast<uint32_t*>(a), w);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < n) a[k] = (uint8_t)(w >> (8 * k));
}

// 4 entries of a block in 8 bits: `top` is the lanes' largest magnitude
template <bool ROOT>
__device__ __forceinline__ uint32_t pack4(const float (&x)[4], const uint32_t (&random)[4], float& scale) {
    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    const uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    const uint32_t e = (uint32_t)max((int)(u >> 23) - 7, 1);
    const float down = __uint_as_float((254u - e) << 23);
    scale = __uint_as_float(e << 23);
    uint32_t w = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t code = e4m3_random(x[k] * down, random[k]);
        if (ROOT) code = x[k] > 0.0f ? max(code, 1u) : code;
        else code |= x[k] < 0.0f ? 0x80u : 0u;
        w |= code << (8 * k);
    }
    return w;
}

template <bool HALF, bool GRAD16, bool PACKED, bool VEC>
__device__ __forceinline__ bool adam_blocks(const AdamwTensor& t, const AdamwHyper& h, int index, long at, int lane) {
    typedef typename std::conditional<GRAD16, bf16_t, float>::type G;
    float p[kAdamUnroll][4], g[kAdamUnroll][4], m[kAdamUnroll][4], v[kAdamUnroll][4];
    uint32_t cm[kAdamUnroll], cv[kAdamUnroll];
    float sm[kAdamUnroll], sv[kAdamUnroll];
    bool bad = false;
#pragma unroll
    for (int q = 0; q < kAdamUnroll; ++q) {
        const long i = at + q * kAdamBlock + lane * 4;
        const int n = (int)max(0l, min(4l, t.n - i));
        load4<VEC>(t.p + i, n, p[q]);
        load4<VEC>(reinterpret_cast<const G*>(t.grad) + i, n, g[q]);
        if (PACKED) {
            cm[q] = load4_codes<VEC>(reinterpret_cast<const uint8_t*>(t.m) + i, n);
            cv[q] = load4_codes<VEC>(reinterpret_cast<const uint8_t*>(t.v) + i, n);
            const long b = at / kAdamBlock + q;
            const bool some = b * kAdamBlock < t.n;
            sm[q] = some ? t.m_scale[b] : 0.0f;
            sv[q] = some ? t.v_scale[b] : 0.0f;
        } else {
            load4<VEC>(reinterpret_cast<const float*>(t.m) + i, n, m[q]);
            load4<VEC>(reinterpret_cast<const float*>(t.v) + i, n, v[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < kAdamUnroll; ++q) {
        const long i = at + q * kAdamBlock + lane * 4;
        const int n = (int)max(0l, min(4l, t.n - i));
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (PACKED) {
                m[q][k] = e4m3_value((cm[q] >> (8 * k)) & 0xffu) * sm[q];
                v[q][k] = e4m3_value((cv[q] >> (8 * k)) & 0x7fu) * sv[q];
            }
            x[k] = adam_entry<PACKED>(h, p[q][k], g[q][k], m[q][k], v[q][k], bad);
        }
        store4<VEC>(t.p + i, n, x);
        if (HALF) store4_half<VEC>(t.half + i, n, x);
        if (PACKED) {
            const uint4 w = philox4x32(h.k0, h.k1, (uint64_t)i / 4, h.T, (uint32_t)index);
            const uint32_t lo[4] = {w.x & 0xffffu, w.y & 0xffffu, w.z & 0xffffu, w.w & 0xffffu};
            const uint32_t hi[4] = {w.x >> 16, w.y >> 16, w.z >> 16, w.w >> 16};
            float a, b;
            const uint32_t wm = pack4<false>(m[q], lo, a), wv = pack4<true>(v[q], hi, b);
            store4_codes<VEC>(reinterpret_cast<uint8_t*>(t.m) + i, n, wm);
            store4_codes<VEC>(reinterpret_cast<uint8_t*>(t.v) + i, n, wv);
            if (lane == 0 && n > 0) {
                t.m_scale[at / kAdamBlock + q] = a;
                t.v_scale[at / kAdamBlock + q] = b;
            }
        } else {
            store4<VEC>(reinterpret_cast<float*>(t.m) + i, n, m[q]);
            store4<VEC>(reinterpret_cast<float*>(t.v) + i, n, v[q]);
        }
    }
    return bad;
}

template <int CAP>
__global__ void __launch_bounds__(kAdamThreads, 3) adamw_kernel(const __grid_constant__ AdamwArgs<CAP> a) {
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
    h.k0 = a.k0; h.k1 = a.k1; h.T = (uint32_t)step + 1u;
    bool bad = false;
    for (unsigned c = blockIdx.x; fine && c < a.chunks; c += gridDim.x) {
        int lo = 0, hi = a.n - 1;   // the last tensor that begins at or before chunk c
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.t[mid].first <= c) lo = mid; else hi = mid - 1;
        }
        const AdamwTensor& t = a.t[lo];
        const long at = (long)(c - t.first) * kAdamChunk + warp * (kAdamUnroll * kAdamBlock);
        if (at >= t.n) continue;
        const int index = a.base + lo;
        switch (t.kind) {
#define SPEC_ADAM_CASE(K)                                                                                   \
    case K:                                                                                                 \
        bad |= adam_blocks<((K) & kAdamHalf) != 0, ((K) & kAdamGradHalf) != 0, ((K) & kAdamPacked) != 0,    \
                           ((K) & kAdamVec) != 0>(t, h, index, at, lane);                                   \
        break;
            SPEC_ADAM_CASE(0) SPEC_ADAM_CASE(1) SPEC_ADAM_CASE(2) SPEC_ADAM_CASE(3)
            SPEC_ADAM_CASE(4) SPEC_ADAM_CASE(5) SPEC_ADAM_CASE(6) SPEC_ADAM_CASE(7)
            SPEC_ADAM_CASE(8) SPEC_ADAM_CASE(9) SPEC_ADAM_CASE(10) SPEC_ADAM_CASE(11)
            SPEC_ADAM_CASE(12) SPEC_ADAM_CASE(13) SPEC_ADAM_CASE(14) SPEC_ADAM_CASE(15)
#undef SPEC_ADAM_CASE
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
    a.k0 = (uint32_t)c.seed;
    a.k1 = (uint32_t)(c.seed >> 32);
    a.status = &reinterpret_cast<WsHeader*>(c.ws)->status;
    a.done = &reinterpret_cast<WsHeader*>(c.ws)->done[0];
    const unsigned most = (unsigned)device_sm_count() * 3u;
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
        const unsigned grid = chunks < most ? (chunks ? (unsigned)chunks : 1u) : most;
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
