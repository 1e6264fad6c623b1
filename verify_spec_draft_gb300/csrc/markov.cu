// markov.cu - the gradients of the Markov bias weights (spec_markov_grad).
//
// The biased rows are z_i = l_i + Wt U[x_i] (x_i the token before position i), so with dz the
// rows' gradient and n = B gamma rows
//     dWt = dz^T Ux          [V, r], Ux the gathered rows U[x_i]       contraction over n
//     dX  = dz Wt            [n, r]                                    contraction over V
//     dU[x] = the sum of dX's rows with x_i = x, in the rows' order
// First the rows' tokens are put in order, with Ux beside them; then the two products, by one pass
// over the weights for a few rows (here) or on the tensor cores (markov_tc.cu); then dX's parts
// are joined into dU's rows.
#include "markov.cuh"

namespace spec {

constexpr int kMarkovThreads = 256;
constexpr int kMarkovWarps = kMarkovThreads / 32;
constexpr int kOrderTile = 2048;                 // tokens compared at a time
constexpr int kOrderCounted = 4096;              // most rows whose order is counted

// The token before row i's position (V: none, or one that is out of range, which is bad).
__device__ __forceinline__ int markov_token(const MarkovParams& p, int i, bool* bad) {
    const int q = i / p.gamma, j = i - q * p.gamma;
    const int t = j == 0 ? p.anchor[q] : p.tokens[(long)q * p.gamma + j - 1];
    if (t < -1 || t >= p.V) *bad = true;
    return t < 0 || t >= p.V ? p.V : t;
}

// The row U[x_i] for the tensor cores, by a warp (0 for a row without a token).
template <typename W>
__device__ __forceinline__ void markov_gather(const MarkovParams& p, const MarkovBind& b, int planes, int n, int i, int token, int lane) {
    const int r8 = round8(p.r);
    const W* u = reinterpret_cast<const W*>(p.U) + (long)token * p.r;
    if (planes == 1 && p.r == r8) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        if (lane < r8 / 8)
            reinterpret_cast<uint4*>(b.ux + (long)i * r8)[lane] = token < p.V ? __ldg(reinterpret_cast<const uint4*>(u) + lane) : zero;
        return;
    }
    for (int k = lane; k < r8; k += 32) {
        float x[3];
        bf16_parts(token < p.V && k < p.r ? load_one(u + k) : 0.0f, x);
#pragma unroll
        for (int q = 0; q < 3; ++q)
            if (q < planes) put<bf16_t>(b.ux, ((long)q * n + i) * r8 + k, x[q]);
    }
}

// Many rows: blocks of kOrderBlock rows are sorted by (token, row) in shared memory, and a row's place is the sum
// of its places among the blocks, found by halving (65,536 rows: some
// 165 us for both kernels, 2385 by counting; 9216 rows 20, 8192 by counting 45; 4096 by counting 16).
constexpr int kOrderBlock = 2048, kOrderMany = 1024;
__global__ void __launch_bounds__(kOrderMany) markov_sort_kernel(MarkovParams p, MarkovBind b, unsigned long long* keys) {
    __shared__ unsigned long long s_key[kOrderBlock];
    const int n = p.B * p.gamma, lo = blockIdx.x * kOrderBlock, tid = threadIdx.x;
    pdl_launch_dependents();
    bool bad = false;
    for (int k = tid; k < kOrderBlock; k += kOrderMany)   // (what is behind the last row comes last)
        s_key[k] = lo + k < n ? ((unsigned long long)markov_token(p, lo + k, &bad) << 32) | (unsigned)(lo + k) : ~0ull;
    if (bad) atomicOr(b.status, SPEC_DEV_TOKEN);
    for (int size = 2; size <= kOrderBlock; size *= 2)
        for (int step = size / 2; step > 0; step /= 2) {
            __syncthreads();
            const int i = tid / step * 2 * step + tid % step, j = i + step;
            const unsigned long long x = s_key[i], y = s_key[j];
            if ((x > y) == ((i & size) == 0)) {
                s_key[i] = y;
                s_key[j] = x;
            }
        }
    __syncthreads();
    for (int k = tid; k < kOrderBlock; k += kOrderMany)
        if (lo + k < n) keys[lo + k] = s_key[k];
}
// keys of a sorted block below `key`
__device__ __forceinline__ int keys_below(const unsigned long long* keys, int m, unsigned long long key) {
    int lo = 0;
    while (m > 0) {
        const int half = m / 2;
        if (keys[lo + half] < key) {
            lo += half + 1;
            m -= half + 1;
        } else {
            m = half;
        }
    }
    return lo;
}
template <typename W>
__global__ void __launch_bounds__(kMarkovThreads) markov_place_kernel(MarkovParams p, MarkovBind b, int planes, const unsigned long long* keys) {
    __shared__ unsigned s_none;
    const int n = p.B * p.gamma, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * kMarkovWarps + warp;
    bool bad = false;
    pdl_launch_dependents();
    const int mine = i < n ? markov_token(p, i, &bad) : 0;
    if (threadIdx.x == 0) s_none = 0u;
    __syncthreads();
    if (i < n) {
        if (lane == 0 && mine >= p.V) atomicOr(&s_none, 1u << warp);
        markov_gather<W>(p, b, planes, n, i, mine, lane);
    }
    pdl_wait_primary();
    if (i < n) {   // a lane takes every 32nd block
        unsigned less = 0u, same = 0u, before = 0u;
        for (int lo = lane * kOrderBlock; lo < n; lo += 32 * kOrderBlock) {
            const int m = min(kOrderBlock, n - lo);
            const unsigned long long first = (unsigned long long)mine << 32;
            const int at = keys_below(keys + lo, m, first), end = keys_below(keys + lo, m, first + (1ull << 32));
            less += (unsigned)at;
            same += (unsigned)(end - at);
            if (lo + kOrderBlock <= i) before += (unsigned)(end - at);
            else if (lo <= i) before += (unsigned)(keys_below(keys + lo, m, first | (unsigned)i) - at);
        }
        less = __reduce_add_sync(0xffffffffu, less);
        same = __reduce_add_sync(0xffffffffu, same);
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) {
            b.order[less + before] = i;
            b.token[less + before] = mine;
            b.run[less + before] = make_int2((int)less, (int)same);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) b.none[blockIdx.x] = (uint8_t)s_none;
}

// Row i's place among the rows by (token, row), counted: n comparisons a row, a warp a row.  The warp
// copies the row U[x_i] for the tensor cores as well; a CTA's 8 rows are a byte of the marks.
template <typename W>
__global__ void __launch_bounds__(kMarkovThreads) markov_order_kernel(MarkovParams p, MarkovBind b, int planes) {
    __shared__ int32_t s_tok[kOrderTile];
    __shared__ unsigned s_none;
    const int n = p.B * p.gamma, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * kMarkovWarps + warp;
    bool bad = false;
    pdl_launch_dependents();
    const int mine = i < n ? markov_token(p, i, &bad) : 0;
    if (threadIdx.x == 0) s_none = 0u;
    __syncthreads();
    if (lane == 0) {
        if (bad) atomicOr(b.status, SPEC_DEV_TOKEN);
        if (i < n && mine >= p.V) atomicOr(&s_none, 1u << warp);
    }
    if (i < n) markov_gather<W>(p, b, planes, n, i, mine, lane);
    int less = 0, same = 0, before = 0;   // tokens below this one, rows of it, those of them before this one
    for (int lo = 0; lo < n; lo += kOrderTile) {
        __syncthreads();
        bool other = false;
#pragma unroll
        for (int k = threadIdx.x; k < kOrderTile; k += kMarkovThreads)
            if (lo + k < n) s_tok[k] = markov_token(p, lo + k, &other);
        __syncthreads();
        const int m = min(kOrderTile, n - lo);
#pragma unroll 4
        for (int k = lane; k < m; k += 32) {
            const int t = s_tok[k];
            less += t < mine ? 1 : 0;
            same += t == mine ? 1 : 0;
            before += t == mine && lo + k < i ? 1 : 0;
        }
    }
    less = (int)__reduce_add_sync(0xffffffffu, (unsigned)less);
    same = (int)__reduce_add_sync(0xffffffffu, (unsigned)same);
    before = (int)__reduce_add_sync(0xffffffffu, (unsigned)before);
    if (i < n && lane == 0) {
        b.order[less + before] = i;
        b.token[less + before] = mine;
        b.run[less + before] = make_int2(less, same);
    }
    if (threadIdx.x == 0) b.none[blockIdx.x] = (uint8_t)s_none;
}

// A few rows: one pass over the vocabulary forms both products.  A thread takes 4 columns of an entry v:
// dWt[v] = sum_i dz[i, v] U[x_i] with U's rows in shared memory, and dX's sums of its columns in
// registers, one per row, which the CTA's threads bring together at the end.  The tensor cores would spend their
// steps of 64 rows on zeros, and need float32 operands split (GPU time of the call, 7 rows, here and there:
// V = 32,000, r = 32 float32 9.9 and 48 us; bf16 weights and outputs at V = 248,320: r = 64 28 and 71, 128 49 and 62,
// 192 73 and 83, 256 91 and 83, with float32 outputs 117 and 126; r = 256 at V = 151,936: 62 and 59, at 32,000: 25 and
// 28).  Bound by memory where V is large, Wt in, dWt and dU's zeros out (5.5 TB/s with float32 outputs), and by
// issue slots beside it; by a chain of latencies where it is small.
// All calls of up to 8 rows come here, the one corner where the other way is 6 to 9 % shorter (r = 256, bf16 outputs,
// large vocabularies) included: a block's gradient then has the same two launches and the same float32 sums
// whatever the rank and the outputs' type.
template <typename T> struct QuadWord { typedef uint2 type; };
template <> struct QuadWord<float> { typedef float4 type; };
__device__ __forceinline__ float4 quad_value(const float4& w) { return w; }
__device__ __forceinline__ float4 quad_value(const uint2& w) {
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
template <bool VEC> __device__ __forceinline__ float4 quad_load(const float* a, int left) {   // entries a[0..3], `left` of them
    if (VEC) return __ldg(reinterpret_cast<const float4*>(a));
    return make_float4(__ldg(a), left > 1 ? __ldg(a + 1) : 0.0f, left > 2 ? __ldg(a + 2) : 0.0f, left > 3 ? __ldg(a + 3) : 0.0f);
}
template <bool VEC> __device__ __forceinline__ uint2 quad_load(const bf16_t* a, int left) {
    if (VEC) return __ldg(reinterpret_cast<const uint2*>(a));
    const unsigned short* h = reinterpret_cast<const unsigned short*>(a);
    uint32_t x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = q < left ? __ldg(h + q) : 0u;
    return make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16);
}
template <bool VEC> __device__ __forceinline__ void quad_store(void* out, int dtype, long at, int left, const float4& x) {
    if (VEC) {
        if (dtype == SPEC_BF16) {
            *reinterpret_cast<uint2*>(reinterpret_cast<bf16_t*>(out) + at) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
        } else {
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at) = x;
        }
        return;
    }
    const float o[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int h = 0; h < 4; ++h)
        if (h < left) put(out, dtype, at + h, o[h]);
}
constexpr int kSmallTurn = 4;                    // most entries of a thread in a turn
constexpr int kSmallTile = 128;                  // most entries of a CTA's turn
// FULL: rows of whole fours, and kSmallTurn entries a turn
template <typename G, typename W, bool FULL>
__global__ void __launch_bounds__(kMarkovThreads, 2) markov_small_kernel(MarkovParams p, MarkovBind b) {
    constexpr int N = kMarkovSmall, K = kSmallTurn, Z = N * kSmallTile / kMarkovThreads;
    __shared__ __align__(16) float s_u[N][SPEC_MAX_RANK];
    __shared__ float s_x[4 * N][kMarkovThreads + 1];     // first, dz's values of two turns
    __shared__ int s_row[N];
    float (*s_z)[N][kSmallTile] = reinterpret_cast<float (*)[N][kSmallTile]>(&s_x[0][0]);
    const int n = p.B * p.gamma, tid = threadIdx.x, pitch = round4(p.r), quads = pitch / 4;
    const int entries = min(kMarkovThreads / quads, kSmallTile);   // side by side
    const int turn = FULL ? K : min(K, kSmallTile / entries), tile = turn * entries;
    const int k = tid % quads * 4, e = tid / quads;
    const W* Wt = reinterpret_cast<const W*>(p.Wt);
    const G* dz = reinterpret_cast<const G*>(p.grad);
    pdl_launch_dependents();
    // the next turn's values are on their way while this one's are used, the first ones' before the tokens are known
    typename QuadWord<W>::type next_w[K];
    G next_z[Z];
    auto fetch = [&](int v0) {
        const int c = tid % kSmallTile, i0 = tid / kSmallTile;
#pragma unroll
        for (int q = 0; q < Z; ++q) {
            const int i = i0 + q * (kMarkovThreads / kSmallTile);
            next_z[q] = G();
            if (i < n && c < tile && v0 + c < p.V) next_z[q] = __ldg(dz + (long)i * p.ld + v0 + c);
        }
#pragma unroll
        for (int q = 0; q < K; ++q) {
            const int v = v0 + q * entries + e;
            next_w[q] = typename QuadWord<W>::type();
            if (e < entries && q < turn && v < p.V) next_w[q] = quad_load<FULL>(Wt + ((long)v * p.r + k), p.r - k);
        }
    };
    const int step = (int)gridDim.x * tile;
    int v0 = (int)blockIdx.x * tile;
    fetch(v0);
    bool bad = false;
    if (tid < N) s_row[tid] = tid < n ? markov_token(p, tid, &bad) : p.V;
    if (bad && blockIdx.x == 0) atomicOr(b.status, SPEC_DEV_TOKEN);
    __syncthreads();
    for (int a = tid; a < N * pitch; a += kMarkovThreads) {
        const int i = a / pitch, c = a - i * pitch;
        s_u[i][c] = s_row[i] < p.V && c < p.r ? load_one(reinterpret_cast<const W*>(p.U) + (long)s_row[i] * p.r + c) : 0.0f;
    }
    float4 x[N], w[K];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int buf = 0; v0 < p.V; v0 += step, buf ^= 1) {
#pragma unroll
        for (int q = 0; q < Z; ++q) {   // (a row without a token counts as 0)
            const int i = tid / kSmallTile + q * (kMarkovThreads / kSmallTile);
            s_z[buf][i][tid % kSmallTile] = s_row[i] < p.V ? to_float(next_z[q]) : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < K; ++q) w[q] = quad_value(next_w[q]);
        __syncthreads();   // (and so the buffer that is written next has been read)
        if (v0 + step < p.V) fetch(v0 + step);
        if (e >= entries) continue;
        float4 o[K];
#pragma unroll
        for (int q = 0; q < K; ++q) o[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float4 u = *reinterpret_cast<const float4*>(&s_u[i][k]);
#pragma unroll
            for (int q = 0; q < K; ++q) {
                if (q >= turn) continue;
                const float z = s_z[buf][i][q * entries + e];
                o[q].x = fmaf(z, u.x, o[q].x); o[q].y = fmaf(z, u.y, o[q].y); o[q].z = fmaf(z, u.z, o[q].z); o[q].w = fmaf(z, u.w, o[q].w);
                x[i].x = fmaf(z, w[q].x, x[i].x); x[i].y = fmaf(z, w[q].y, x[i].y);
                x[i].z = fmaf(z, w[q].z, x[i].z); x[i].w = fmaf(z, w[q].w, x[i].w);
            }
        }
#pragma unroll
        for (int q = 0; q < K; ++q) {
            const int v = v0 + q * entries + e;
            if (q >= turn || v >= p.V) continue;
            quad_store<FULL>(p.dWt_out, p.odt, (long)v * p.r + k, p.r - k, o[q]);
            quad_store<FULL>(p.dU_out, p.odt, (long)v * p.r + k, p.r - k, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        }
    }
    __syncthreads();
    // the threads' sums of dX, in order
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s_x[4 * i][tid] = x[i].x;
        s_x[4 * i + 1][tid] = x[i].y;
        s_x[4 * i + 2][tid] = x[i].z;
        s_x[4 * i + 3][tid] = x[i].w;
    }
    __syncthreads();
    for (int a = tid; a < n * pitch; a += kMarkovThreads) {
        const int i = a / pitch, c = a - i * pitch;
        const float* from = &s_x[4 * i + (c & 3)][c >> 2];
        float s = 0.0f;
#pragma unroll 4
        for (int q = 0; q < entries; ++q) s += from[q * quads];
        b.part[((long)blockIdx.x * n + i) * pitch + c] = s;
    }
}

// dU's rows: the CTA at every kJoinRun-th of a token's ordered rows sums the parts of that many; where
// they are all, that is dU's row, otherwise the sum is kept for markov_runs_kernel.  16-byte columns go over
// lanes and the parts over groups of threads, whose sums meet in order.
constexpr int kJoinThreads = 256;
constexpr int kJoinMany = 1024;                  // of the few rows' many parts
__device__ __forceinline__ void join_out(const MarkovParams& p, int t, int k, const float4& s) {
    const float o[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int h = 0; h < 4; ++h)
        if (4 * k + h < p.r) put(p.dU_out, p.odt, (long)t * p.r + 4 * k + h, o[h]);
}
__device__ __forceinline__ bool join_meet(float4* s_sum, float4& s, int k, int g, int quads, int groups) {
    if (g < groups) s_sum[g * quads + k] = s;
    __syncthreads();
    if (g != 0) return false;
    for (int q = 1; q < groups; ++q) {
        const float4 x = s_sum[q * quads + k];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    return true;
}
template <bool SMALL>   // (kMarkovSmall rows at most: their order is found here)
__global__ void __launch_bounds__(SMALL ? kJoinMany : kJoinThreads) markov_join_kernel(MarkovParams p, MarkovBind b, MarkovJoin a) {
    constexpr int TH = SMALL ? kJoinMany : kJoinThreads;
    __shared__ float4 s_sum[TH];
    const int at = blockIdx.x;
    int t, rows, all, index[kJoinRun];
    pdl_launch_dependents();
    if (!SMALL) pdl_wait_primary();
    if (SMALL) {
        static_assert(kMarkovSmall == kJoinRun, "a CTA joins all rows of a token");
        const int n = p.B * p.gamma;
        bool bad = false;
        t = markov_token(p, at, &bad);
        rows = 0;
        int first = at;
#pragma unroll
        for (int i = kMarkovSmall - 1; i >= 0; --i)
            if (i < n && markov_token(p, i, &bad) == t) first = i;
#pragma unroll
        for (int i = 0; i < kMarkovSmall; ++i) {
            if (i >= n || markov_token(p, i, &bad) != t) continue;
#pragma unroll
            for (int q = 0; q < kJoinRun; ++q)
                if (q == rows) index[q] = i;
            ++rows;
        }
        all = rows;
        pdl_wait_primary();
        if (t >= p.V || first < at) return;   // none, or that one's
    } else {
        const int2 run = b.run[at];
        t = b.token[at];
        if ((at - run.x) % kJoinRun != 0) return;
        rows = min(kJoinRun, run.x + run.y - at);
        all = run.y;
#pragma unroll
        for (int q = 0; q < kJoinRun; ++q) index[q] = b.order[at + min(q, rows - 1)];
    }
    const int quads = round4(p.r) / 4, groups = TH / quads;
    const int k = threadIdx.x % quads, g = threadIdx.x / quads;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (g < groups) {
#pragma unroll 2
        for (int part = g; part < a.parts; part += groups)
#pragma unroll
            for (int q = 0; q < kJoinRun; ++q) {
                if (q >= rows) continue;
                const float4 x = *reinterpret_cast<const float4*>(b.part + (part * a.part_stride + index[q]) * a.pitch + 4 * k);
                s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
            }
    }
    if (!join_meet(s_sum, s, k, g, quads, groups)) return;
    if (!SMALL && t >= p.V) {   // rows without a token: nothing but whether they are finite
        if (!(fabsf(s.x + s.y + s.z + s.w) < INFINITY)) *(volatile unsigned*)b.unclean = 1u;
        return;
    }
    if (all <= kJoinRun) join_out(p, t, k, s);
    else reinterpret_cast<float4*>(b.runs + (long)at * round4(p.r))[k] = s;
}
cudaError_t markov_join(const MarkovParams& p, const MarkovBind& b, const MarkovJoin& a, cudaStream_t stream) {
    return launch_behind(markov_join_kernel<false>, dim3((unsigned)(p.B * p.gamma)), kJoinThreads, 0, stream, p, b, a);
}

// The tokens of more rows: a CTA looks at 32 places for where one begins.
__global__ void __launch_bounds__(kJoinThreads) markov_runs_kernel(MarkovParams p, MarkovBind b) {
    __shared__ float4 s_sum[kJoinThreads];
    pdl_wait_primary();
    if (blockIdx.x == 0 && threadIdx.x == 0) *b.unclean = 0u;
    const int n = p.B * p.gamma;
    const int quads = round4(p.r) / 4, groups = kJoinThreads / quads;
    const int k = threadIdx.x % quads, g = threadIdx.x / quads;
    const int mine = blockIdx.x * 32 + (threadIdx.x & 31);
    const int2 look = mine < n && b.token[mine] < p.V ? b.run[mine] : make_int2(-1, 0);
    unsigned found = __ballot_sync(0xffffffffu, look.x == mine && look.y > kJoinRun);
    for (; found; found &= found - 1) {
        const int at = blockIdx.x * 32 + __ffs(found) - 1;
        const int t = b.token[at], terms = (b.run[at].y + kJoinRun - 1) / kJoinRun;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (g < groups) {
            const int lo = terms * g / groups, hi = (int)((long)terms * (g + 1) / groups);
#pragma unroll 8
            for (int e = lo; e < hi; ++e) {
                const float4 x = reinterpret_cast<const float4*>(b.runs + (long)(at + e * kJoinRun) * round4(p.r))[k];
                s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
            }
        }
        if (join_meet(s_sum, s, k, g, quads, groups)) join_out(p, t, k, s);
        __syncthreads();
    }
}

static size_t markov_bind(MarkovBind& b, void* ws, int n, int r, int V) {
    uint8_t* w = reinterpret_cast<uint8_t*>(ws);
    b.status = &reinterpret_cast<WsHeader*>(ws)->status;
    b.unclean = &reinterpret_cast<WsHeader*>(ws)->done[0];
    size_t at = kWsHeaderBytes;
    auto take = [&](size_t bytes) {
        uint8_t* q = w + at;
        at += align256(bytes);
        return q;
    };
    b.order = reinterpret_cast<int32_t*>(take((size_t)n * 4));
    b.token = reinterpret_cast<int32_t*>(take((size_t)n * 4));
    b.run = reinterpret_cast<int2*>(take((size_t)n * 8));
    b.runs = reinterpret_cast<float*>(take((size_t)n * round4(r) * 4));
    const int columns = markov_slice(n, r, V);
    b.none = take((size_t)(n + 63) / 64 * 8);
    b.ux = reinterpret_cast<bf16_t*>(take((size_t)3 * n * round8(r) * 2));
    const int tiles = (n + 255) / 256;
    // (a few rows' slabs are less: kMarkovSlabs n r of them)
    static_assert(kMarkovSlabs * kMarkovSmall <= kMarkovItems * 128, "room for the slabs' parts");
    b.part = reinterpret_cast<float*>(take((size_t)(tiles > kMarkovItems ? tiles : kMarkovItems) * 256 * (r > 128 ? 256 : 128) * 4));
    b.stage_bytes = (size_t)6 * (n + round8(r)) * round8(columns) + 4096;
    b.stage = reinterpret_cast<bf16_t*>(take(b.stage_bytes));
    return at;
}

size_t markov_grad_workspace_bytes(int B, int gamma, int V, int r) {
    MarkovBind b;
    return markov_bind(b, nullptr, B * gamma, r, V);
}

template <typename G, typename W>
static int markov_small_launch(const MarkovParams& p, const MarkovBind& b, cudaStream_t stream) {
    const int side = kMarkovThreads / (round4(p.r) / 4), entries = side < kSmallTile ? side : kSmallTile;
    const int tile = entries * (kSmallTile / entries < kSmallTurn ? kSmallTile / entries : kSmallTurn);
    int slabs = (p.V + tile - 1) / tile;
    const int most = 2 * device_sm_count() < kMarkovSlabs ? 2 * device_sm_count() : kMarkovSlabs;
    if (slabs > most) slabs = most;
    if (p.r % 4 == 0 && tile == entries * kSmallTurn) markov_small_kernel<G, W, true><<<slabs, kMarkovThreads, 0, stream>>>(p, b);
    else markov_small_kernel<G, W, false><<<slabs, kMarkovThreads, 0, stream>>>(p, b);
    return slabs;
}

cudaError_t markov_grad_launch(const MarkovParams& p, void* ws, cudaStream_t stream) {
    const int n = p.B * p.gamma;
    MarkovBind b;
    markov_bind(b, ws, n, p.r, p.V);
    const bool small = n <= kMarkovSmall, g16 = p.gdt == SPEC_BF16, w16 = p.wdt == SPEC_BF16;
    if (small) {
        MarkovJoin join = {0, n, round4(p.r)};
        join.parts = g16 ? (w16 ? markov_small_launch<bf16_t, bf16_t>(p, b, stream) : markov_small_launch<bf16_t, float>(p, b, stream))
                         : (w16 ? markov_small_launch<float, bf16_t>(p, b, stream) : markov_small_launch<float, float>(p, b, stream));
        const cudaError_t e = launch_behind(markov_join_kernel<true>, dim3((unsigned)n), kJoinMany, 0, stream, p, b, join);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const unsigned grid = (unsigned)((n + 63) / 64) * (64 / kMarkovWarps);   // whole words of marks
    cudaError_t e = cudaSuccess;
    if (n > kOrderCounted) {
        unsigned long long* keys = reinterpret_cast<unsigned long long*>(b.runs);   // (not in use yet; 16 bytes a row at least)
        markov_sort_kernel<<<(n + kOrderBlock - 1) / kOrderBlock, kOrderMany, 0, stream>>>(p, b, keys);
        e = w16 ? launch_behind(markov_place_kernel<bf16_t>, dim3(grid), dim3(kMarkovThreads), 0, stream, p, b, 1, keys)
                : launch_behind(markov_place_kernel<float>, dim3(grid), dim3(kMarkovThreads), 0, stream, p, b, 3, keys);
    } else if (w16) {
        markov_order_kernel<bf16_t><<<grid, kMarkovThreads, 0, stream>>>(p, b, 1);
    } else {
        markov_order_kernel<float><<<grid, kMarkovThreads, 0, stream>>>(p, b, 3);
    }
    if (e == cudaSuccess) e = markov_tc_launch(p, b, stream);
    if (e == cudaSuccess) e = launch_behind(markov_runs_kernel, dim3((unsigned)((n + 31) / 32)), kJoinThreads, 0, stream, p, b);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spec
