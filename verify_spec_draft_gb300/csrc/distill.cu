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
// Weights are 2^((z - m) log2e / t) with m the row's maximum, taken from z before the
// scaling, so that rows filled with the type's lowest value neither overflow nor vanish.
// Logarithms of p and q are differences from the two maxima, so the loss keeps float32's
// absolute accuracy whatever the logits' offset.
#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kDistThreads = 256;
constexpr int kDistWarps = kDistThreads / 32;
constexpr int kDistWords = 8;                              // words a thread holds
constexpr int kDistPiece = kDistThreads * kDistWords;      // words of a CTA

__host__ __device__ inline int distill_pieces(int V, int elt_bytes) {
    const int E = 16 / elt_bytes;
    return ((V + 2 * E - 2) / E + kDistPiece - 1) / kDistPiece;
}

// Statistics of the entries that no id names, per piece.
template <typename T>
__global__ void __launch_bounds__(kDistThreads) distill_scan_kernel(DistillParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    __shared__ uint32_t s_named[kDistPiece * E / 32];
    __shared__ float2 s_run[kDistWarps];
    const int row = blockIdx.x / p.pieces, piece = blockIdx.x - row * p.pieces;
    if (p.weight && p.weight[row] == 0.0f) return;
    const int tid = threadIdx.x;
    const RowWords<T> in(reinterpret_cast<const T*>(p.student) + (long)row * p.ld, p.V);
    const int w0 = piece * kDistPiece;
    const uint32_t ninf = NegInf<T>::word;
    uint4 w[kDistWords];
#pragma unroll
    for (int q = 0; q < kDistWords; ++q) {
        const int i = w0 + q * kDistThreads + tid;
        w[q] = i < in.n ? in.load(i) : make_uint4(ninf, ninf, ninf, ninf);
    }
    for (int i = tid; i < kDistPiece * E / 32; i += kDistThreads) s_named[i] = 0u;
    __syncthreads();
    const int e0 = in.entry(w0);
    for (int k = tid; k < p.K; k += kDistThreads) {
        const int id = p.ids[(long)row * p.K + k];
        const unsigned at = (unsigned)(id - e0);
        if (id >= 0 && id < p.V && at < (unsigned)(kDistPiece * E)) atomicOr(&s_named[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < kDistWords; ++q) {
        const int at = (q * kDistThreads + tid) * E;
        const uint32_t named = (s_named[at >> 5] >> (at & 31)) & ((1u << E) - 1u);
        if (named) {
            uint32_t h[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
            for (int k = 0; k < E; ++k) {
                if (!((named >> k) & 1u)) continue;
                if (sizeof(T) == 2) h[k >> 1] = (h[k >> 1] & ((k & 1) ? 0x0000ffffu : 0xffff0000u)) | ((k & 1) ? 0xff800000u : 0xff80u);
                else h[k & 3] = 0xff800000u;
            }
            w[q] = make_uint4(h[0], h[1], h[2], h[3]);
        }
        m = f_max_nan(m, u4_max_nan<sizeof(T)>(w[q]));
    }
    // a NaN or +inf shows in the maximum
    float s = 0.0f;
    if (m > -INFINITY) {
#pragma unroll
        for (int q = 0; q < kDistWords; ++q)
#pragma unroll
            for (int k = 0; k < E; ++k) s += ex2((word_entry<T>(w[q], k) - m) * p.scale);
    }
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = f_max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    s = warp_sum(m == -INFINITY ? 0.0f : s * ex2((m - M) * p.scale));
    if ((tid & 31) == 0) s_run[tid >> 5] = make_float2(M, s);
    __syncthreads();
    if (tid == 0) {
        float CM = -INFINITY, cs = 0.0f;
        for (int i = 0; i < kDistWarps; ++i) CM = f_max_nan(CM, s_run[i].x);
        for (int i = 0; i < kDistWarps; ++i)
            if (s_run[i].x != -INFINITY) cs += s_run[i].y * ex2((s_run[i].x - CM) * p.scale);
        p.parts[(long)row * p.pieces + piece] = make_float2(CM, cs);
    }
}

// One CTA per row: merges the pieces, forms the loss and what the gradient needs.
__device__ __forceinline__ float cta_max_nan(float x, float* s_f) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = f_max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_f[threadIdx.x >> 5] = x;
    __syncthreads();
    x = s_f[0];
    for (int i = 1; i < SPEC_MAX_TEACHER / 32; ++i) x = f_max_nan(x, s_f[i]);
    return x;
}
__device__ __forceinline__ float cta_sum_f(float x, float* s_f) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_f[threadIdx.x >> 5] = x;
    __syncthreads();
    x = s_f[0];
    for (int i = 1; i < SPEC_MAX_TEACHER / 32; ++i) x += s_f[i];
    return x;
}

template <typename T>
__global__ void __launch_bounds__(SPEC_MAX_TEACHER) distill_finish_kernel(DistillParams p) {
    __shared__ float s_f[SPEC_MAX_TEACHER / 32];
    __shared__ int s_id[SPEC_MAX_TEACHER];
    const int row = blockIdx.x, tid = threadIdx.x;
    const float wt = p.weight ? p.weight[row] : 1.0f;
    float4* st = p.stats + row;
    if (wt == 0.0f) {   // the row does not count and is not read
        if (tid == 0) {
            p.loss_out[row] = 0.0f;
            if (p.lse_out) p.lse_out[row] = 0.0f;
            *st = make_float4(0.0f, 0.0f, 1.0f, 0.0f);
        }
        return;
    }
    const T* zr = reinterpret_cast<const T*>(p.student) + (long)row * p.ld;
    int id = -1;
    float a = -INFINITY, z = -INFINITY;
    if (tid < p.K) {
        const long at = (long)row * p.K + tid;
        id = p.ids[at];
        a = p.values_dtype == SPEC_BF16 ? to_float(reinterpret_cast<const bf16_t*>(p.values)[at])
                                        : reinterpret_cast<const float*>(p.values)[at];
    }
    s_id[tid] = id;
    __syncthreads();
    bool bad_id = id < -1 || id >= p.V;
    if (id >= 0)
        for (int k = 0; k < tid; ++k) bad_id |= s_id[k] == id;
    if (id < 0 || bad_id) a = -INFINITY;
    else z = to_float(zr[id]);
    const float at = p.tail ? p.tail[row] : -INFINITY;
    const int nbad = __syncthreads_count(bad_id);
    // student
    float m = z;
    for (int i = tid; i < p.pieces; i += SPEC_MAX_TEACHER) m = f_max_nan(m, p.parts[(long)row * p.pieces + i].x);
    const float M = cta_max_nan(m, s_f);
    float ss = 0.0f;
    for (int i = tid; i < p.pieces; i += SPEC_MAX_TEACHER) {
        const float2 ms = p.parts[(long)row * p.pieces + i];
        if (ms.x != -INFINITY) ss += ms.y * ex2((ms.x - M) * p.scale);
    }
    const bool no_row = !(M < INFINITY) || M == -INFINITY;
    const float qe = no_row ? 0.0f : ex2((z - M) * p.scale);   // 0 for an absent entry
    const float ST = cta_sum_f(ss, s_f);
    const float Z = ST + cta_sum_f(qe, s_f);
    // teacher, in units of 1 (the tail's)
    const float top = cta_max_nan(f_max_nan(a * p.inv_t, at), s_f);
    const bool taught = top != -INFINITY, bad_row = no_row || !(top < INFINITY) || !(fabsf(wt) < INFINITY);
    const float ak = taught ? fmaf(a, p.inv_t, -top) : -INFINITY, aT = taught ? at - top : -INFINITY;
    const float P = cta_sum_f(__expf(ak), s_f) + __expf(aT);
    const float lP = logf(P), lZ = logf(Z);
    const float pk = taught ? __expf(ak) / P : 0.0f, pT = taught ? __expf(aT) / P : 0.0f;
    float l = pk > 0.0f ? pk * ((ak - lP) - ((z - M) * p.inv_t - lZ)) : 0.0f;
    if (tid == 0 && pT > 0.0f) l += pT * ((aT - lP) - (logf(ST) - lZ));
    const float loss = cta_sum_f(l, s_f);
    const float g = wt * p.inv_t;
    const bool bad = bad_row || nbad > 0;
    if (p.grad_out && tid < p.K) {
        const float d = taught ? (qe / Z - pk) * g : 0.0f;
        p.named_grad[(long)row * p.K + tid] = bad ? NAN : d;
    }
    if (tid == 0) {
        p.loss_out[row] = bad ? NAN : loss;
        if (p.lse_out) p.lse_out[row] = bad ? NAN : fmaf(M, p.inv_t, lZ);
        const float cT = taught ? g * (1.0f / Z - (ST > 0.0f ? pT / ST : 0.0f)) : 0.0f;
        *st = make_float4(bad ? 0.0f : M, bad ? NAN : cT, 0.0f, 0.0f);
        if (nbad) atomicOr(p.status, SPEC_DEV_TOKEN);
        if (bad_row) atomicOr(p.status, SPEC_DEV_NONFINITE);
    }
}

// The gradient: the weight times the row's coefficient, then the named entries.
template <typename T>
__global__ void __launch_bounds__(kDistThreads) distill_grad_kernel(DistillParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    const int row = blockIdx.x / p.pieces, piece = blockIdx.x - row * p.pieces;
    const int tid = threadIdx.x;
    const RowWords<T> in(reinterpret_cast<const T*>(p.student) + (long)row * p.ld, p.V);
    T* out = reinterpret_cast<T*>(p.grad_out) + (long)row * p.ld;
    const int w0 = piece * kDistPiece;
    const float4 st = p.stats[row];
    const bool skip = st.z != 0.0f, nan = isnan(st.y);
    uint4 w[kDistWords];
#pragma unroll
    for (int q = 0; q < kDistWords; ++q) {
        const int i = w0 + q * kDistThreads + tid;
        if (i < in.n && !skip) w[q] = in.load(i);
    }
#pragma unroll
    for (int q = 0; q < kDistWords; ++q) {
        const int i = w0 + q * kDistThreads + tid;
        if (i >= in.n) continue;
        float d[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
            d[k] = skip ? 0.0f : ex2((word_entry<T>(w[q], k) - st.x) * p.scale) * st.y;
            if (nan) d[k] = NAN;
        }
        in.store(out, i, word_of<T>(d));
    }
    if (skip || nan) return;
    __syncthreads();   // the piece is written; its named entries replace what is there
    const int e0 = in.entry(w0);
    for (int k = tid; k < p.K; k += kDistThreads) {
        const int id = p.ids[(long)row * p.K + k];
        if (id < 0 || (unsigned)(id - e0) >= (unsigned)(kDistPiece * E)) continue;
        const float d = p.named_grad[(long)row * p.K + k];
        if (sizeof(T) == 2) out[id] = (T)__bfloat16_as_ushort(__float2bfloat16_rn(d));
        else out[id] = (T)d;
    }
}

static size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t distill_workspace_bytes(int rows, int K, int V) {
    return kWsHeaderBytes + align256((size_t)rows * sizeof(float4)) +
           align256((size_t)rows * distill_pieces(V, 4) * sizeof(float2)) + align256((size_t)rows * K * sizeof(float));
}

template <typename T>
static cudaError_t distill_typed(DistillParams p, cudaStream_t stream) {
    p.pieces = distill_pieces(p.V, sizeof(T));
    const long grid = (long)p.rows * p.pieces;
    if (grid > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    distill_scan_kernel<T><<<(unsigned)grid, kDistThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    distill_finish_kernel<T><<<p.rows, SPEC_MAX_TEACHER, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.grad_out) return e;
    distill_grad_kernel<T><<<(unsigned)grid, kDistThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t distill_launch(DistillParams p, void* ws, cudaStream_t stream) {
    p.status = &reinterpret_cast<WsHeader*>(ws)->status;
    uint8_t* b = reinterpret_cast<uint8_t*>(ws) + kWsHeaderBytes;
    p.stats = reinterpret_cast<float4*>(b);
    b += align256((size_t)p.rows * sizeof(float4));
    p.parts = reinterpret_cast<float2*>(b);
    b += align256((size_t)p.rows * distill_pieces(p.V, 4) * sizeof(float2));
    p.named_grad = reinterpret_cast<float*>(b);
    return p.dtype == SPEC_BF16 ? distill_typed<bf16_t>(p, stream) : distill_typed<float>(p, stream);
}

}  // namespace spec
