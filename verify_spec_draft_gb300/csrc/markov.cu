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

// The token before row i's position (V: none, or one that is out of range, which is bad).
__device__ __forceinline__ int markov_token(const MarkovParams& p, int i, bool* bad) {
    const int q = i / p.gamma, j = i - q * p.gamma;
    const int t = j == 0 ? p.anchor[q] : p.tokens[(long)q * p.gamma + j - 1];
    if (t < -1 || t >= p.V) *bad = true;
    return t < 0 || t >= p.V ? p.V : t;
}

// Row i's place among the rows by (token, row), counted: n comparisons a row, a warp a row.  The warp
// copies the row U[x_i] for the tensor cores as well; a CTA's 8 rows are a byte of the marks.
template <typename W>
__global__ void __launch_bounds__(kMarkovThreads) markov_order_kernel(MarkovParams p, MarkovBind b, int planes) {
    __shared__ int32_t s_tok[kOrderTile];
    __shared__ unsigned s_none;
    const int n = p.B * p.gamma, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * kMarkovWarps + warp, r8 = round8(p.r);
    bool bad = false;
    const int mine = i < n ? markov_token(p, i, &bad) : 0;
    if (threadIdx.x == 0) s_none = 0u;
    __syncthreads();
    if (lane == 0) {
        if (bad) atomicOr(b.status, SPEC_DEV_TOKEN);
        if (i < n && mine >= p.V) atomicOr(&s_none, 1u << warp);
    }
    if (i < n) {
        const W* u = reinterpret_cast<const W*>(p.U) + (long)mine * p.r;
        if (planes == 1 && p.r == r8) {
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            if (lane < r8 / 8)
                reinterpret_cast<uint4*>(b.ux + (long)i * r8)[lane] = mine < p.V ? __ldg(reinterpret_cast<const uint4*>(u) + lane) : zero;
        } else {
            for (int k = lane; k < r8; k += 32) {
                float x[3];
                bf16_parts(mine < p.V && k < p.r ? load_one(u + k) : 0.0f, x);
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    if (q < planes) put<bf16_t>(b.ux, ((long)q * n + i) * r8 + k, x[q]);
            }
        }
    }
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

// A few rows: one pass over the vocabulary forms both products.  A warp takes an entry v, its lanes
// the r columns: dWt[v] = sum_i dz[i, v] U[x_i] with the rows' U in registers, and dX's sums, one per row
// and column, in registers too.  Bound by memory: Wt in, dWt and dU's zeros out.  7 rows, the tensor cores
// would spend their steps of 64 rows on zeros.
template <typename G, typename W, int C>
__global__ void __launch_bounds__(kMarkovThreads) markov_small_kernel(MarkovParams p, MarkovBind b) {
    constexpr int N = kMarkovSmall, kV = kMarkovTurn;
    __shared__ __align__(16) float s_d[kV][N];
    __shared__ float s_x[kMarkovWarps][32 * C];
    __shared__ int s_row[N];
    const int n = p.B * p.gamma, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad = false;
    if (tid < N) s_row[tid] = tid < n ? markov_token(p, tid, &bad) : p.V;
    if (bad && blockIdx.x == 0) atomicOr(b.status, SPEC_DEV_TOKEN);
    __syncthreads();
    const G* dz = reinterpret_cast<const G*>(p.grad);
    float u[N][C], x[N][C];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = c * 32 + lane;
            x[i][c] = 0.0f;
            u[i][c] = s_row[i] < p.V && k < p.r ? load_one(reinterpret_cast<const W*>(p.U) + (long)s_row[i] * p.r + k) : 0.0f;
        }
    const int turns = (p.V + kV - 1) / kV;
    for (int turn = blockIdx.x; turn < turns; turn += gridDim.x) {
        const int v0 = turn * kV;
        __syncthreads();
        for (int e = tid; e < kV * N; e += kMarkovThreads) {
            const int i = e / kV, v = v0 + e % kV;
            s_d[e % kV][i] = v < p.V && s_row[i] < p.V ? load_one(dz + (long)i * p.ld + v) : 0.0f;
        }
        __syncthreads();
#pragma unroll 4
        for (int e = warp; e < kV; e += kMarkovWarps) {
            const int v = v0 + e;
            if (v >= p.V) break;
            float w[C], o[C], d[N];
            *reinterpret_cast<float4*>(d) = *reinterpret_cast<const float4*>(&s_d[e][0]);
            *reinterpret_cast<float4*>(d + 4) = *reinterpret_cast<const float4*>(&s_d[e][4]);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = c * 32 + lane;
                w[c] = k < p.r ? load_one(reinterpret_cast<const W*>(p.Wt) + (long)v * p.r + k) : 0.0f;
                o[c] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    o[c] = fmaf(d[i], u[i][c], o[c]);
                    x[i][c] = fmaf(d[i], w[c], x[i][c]);
                }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = c * 32 + lane;
                if (k >= p.r) continue;
                put(p.dWt_out, p.odt, (long)v * p.r + k, o[c]);
                put(p.dU_out, p.odt, (long)v * p.r + k, 0.0f);
            }
        }
    }
    // the warps' sums of dX, in order
    const int pitch = round4(p.r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) s_x[warp][c * 32 + lane] = x[i][c];
        __syncthreads();
        if (i < n && tid < pitch) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kMarkovWarps; ++q) s += tid < 32 * C ? s_x[q][tid] : 0.0f;
            b.part[((long)blockIdx.x * n + i) * pitch + tid] = s;
        }
    }
}

// dU's rows: the CTA at every kJoinRun-th of a token's ordered rows sums the parts of that many; where
// they are all, that is dU's row, otherwise the sum is kept for markov_runs_kernel.  16-byte columns go over
// lanes and the parts over groups of threads, whose sums meet in order.
constexpr int kJoinThreads = 256;
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
__global__ void __launch_bounds__(kJoinThreads) markov_join_kernel(MarkovParams p, MarkovBind b, MarkovJoin a) {
    __shared__ float4 s_sum[kJoinThreads];
    const int at = blockIdx.x;
    int t, rows, all, index[kJoinRun];
    if (SMALL) {
        static_assert(kMarkovSmall == kJoinRun, "a CTA joins all rows of a token");
        const int n = p.B * p.gamma;
        bool bad = false;
        t = markov_token(p, at, &bad);
        rows = 0;
#pragma unroll
        for (int i = 0; i < kMarkovSmall; ++i) {
            if (i >= n || markov_token(p, i, &bad) != t) continue;
            if (i < at) return;   // that one's
#pragma unroll
            for (int q = 0; q < kJoinRun; ++q)
                if (q == rows) index[q] = i;
            ++rows;
        }
        all = rows;
    } else {
        const int2 run = b.run[at];
        t = b.token[at];
        if ((at - run.x) % kJoinRun != 0) return;
        rows = min(kJoinRun, run.x + run.y - at);
        all = run.y;
#pragma unroll
        for (int q = 0; q < kJoinRun; ++q) index[q] = b.order[at + min(q, rows - 1)];
    }
    if (SMALL && t >= p.V) return;
    const int quads = round4(p.r) / 4, groups = kJoinThreads / quads;
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
void markov_join(const MarkovParams& p, const MarkovBind& b, const MarkovJoin& a, cudaStream_t stream) {
    markov_join_kernel<false><<<p.B * p.gamma, kJoinThreads, 0, stream>>>(p, b, a);
}

// The tokens of more rows: a CTA looks at 32 places for where one begins.
__global__ void __launch_bounds__(kJoinThreads) markov_runs_kernel(MarkovParams p, MarkovBind b) {
    __shared__ float4 s_sum[kJoinThreads];
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

// (the sums' registers grow with r: 5 rows of r = 256 take 285 us here, 140 on the tensor cores)
static bool markov_small(int n, int r) { return n <= kMarkovSmall && r <= 64; }

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
    if (markov_small(n, r)) {
        b.part = reinterpret_cast<float*>(take((size_t)kMarkovSlabs * n * round4(r) * 4));
        return at;
    }
    b.order = reinterpret_cast<int32_t*>(take((size_t)n * 4));
    b.token = reinterpret_cast<int32_t*>(take((size_t)n * 4));
    b.run = reinterpret_cast<int2*>(take((size_t)n * 8));
    b.runs = reinterpret_cast<float*>(take((size_t)n * round4(r) * 4));
    const int columns = markov_slice(n, r, V);
    b.none = take((size_t)(n + 63) / 64 * 8);
    b.ux = reinterpret_cast<bf16_t*>(take((size_t)3 * n * round8(r) * 2));
    const int tiles = (n + 255) / 256;
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
    int slabs = (p.V + kMarkovTurn - 1) / kMarkovTurn;
    const int most = 2 * device_sm_count() < kMarkovSlabs ? 2 * device_sm_count() : kMarkovSlabs;
    if (slabs > most) slabs = most;
    if (p.r <= 32) markov_small_kernel<G, W, 1><<<slabs, kMarkovThreads, 0, stream>>>(p, b);
    else markov_small_kernel<G, W, 2><<<slabs, kMarkovThreads, 0, stream>>>(p, b);
    return slabs;
}

cudaError_t markov_grad_launch(const MarkovParams& p, void* ws, cudaStream_t stream) {
    const int n = p.B * p.gamma;
    MarkovBind b;
    markov_bind(b, ws, n, p.r, p.V);
    const bool small = markov_small(n, p.r), g16 = p.gdt == SPEC_BF16, w16 = p.wdt == SPEC_BF16;
    if (small) {
        MarkovJoin join = {0, n, round4(p.r)};
        join.parts = g16 ? (w16 ? markov_small_launch<bf16_t, bf16_t>(p, b, stream) : markov_small_launch<bf16_t, float>(p, b, stream))
                         : (w16 ? markov_small_launch<float, bf16_t>(p, b, stream) : markov_small_launch<float, float>(p, b, stream));
        markov_join_kernel<true><<<n, kJoinThreads, 0, stream>>>(p, b, join);
        return cudaGetLastError();
    }
    const unsigned grid = (unsigned)((n + 63) / 64) * (64 / kMarkovWarps);   // whole words of marks
    if (w16) markov_order_kernel<bf16_t><<<grid, kMarkovThreads, 0, stream>>>(p, b, 1);
    else markov_order_kernel<float><<<grid, kMarkovThreads, 0, stream>>>(p, b, 3);
    const cudaError_t e = markov_tc_launch(p, b, stream);
    if (e != cudaSuccess) return e;
    markov_runs_kernel<<<(n + 31) / 32, kJoinThreads, 0, stream>>>(p, b);
    return cudaGetLastError();
}

}  // namespace spec
