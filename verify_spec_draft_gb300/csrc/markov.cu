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

// Row i's place among the rows by (token, row), counted: n comparisons a row, a warp a row.  A
// second half of the grid copies the rows U[x_i] for the tensor cores and marks the rows without
// a token.
template <typename W>
__global__ void __launch_bounds__(kMarkovThreads) markov_order_kernel(MarkovParams p, MarkovBind b, int planes) {
    __shared__ int32_t s_tok[kOrderTile];
    const int n = p.B * p.gamma, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto token_of = [&](int i, bool* bad) {
        const int q = i / p.gamma, j = i - q * p.gamma;
        const int t = j == 0 ? p.anchor[q] : p.tokens[(long)q * p.gamma + j - 1];
        if (t < -1 || t >= p.V) *bad = true;
        return t < 0 || t >= p.V ? p.V : t;
    };
    bool bad = false;
    const int ranks = (n + kMarkovWarps - 1) / kMarkovWarps;
    if ((int)blockIdx.x >= ranks) {   // (a CTA of 64 rows, so that it has a whole word of marks)
        const int i0 = ((int)blockIdx.x - ranks) * 64, r8 = round8(p.r);
        if (warp == 0) {
            const unsigned lo = __ballot_sync(0xffffffffu, i0 + lane < n && token_of(i0 + lane, &bad) >= p.V);
            const unsigned hi = __ballot_sync(0xffffffffu, i0 + 32 + lane < n && token_of(i0 + 32 + lane, &bad) >= p.V);
            if (lane == 0) b.none[i0 >> 6] = (unsigned long long)hi << 32 | lo;
        }
        for (int i = i0 + warp; i < min(n, i0 + 64); i += kMarkovWarps) {
            const int t = token_of(i, &bad);
            const W* u = reinterpret_cast<const W*>(p.U) + (long)t * p.r;
            if (planes == 1 && p.r == r8) {
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                if (lane < r8 / 8)
                    reinterpret_cast<uint4*>(b.ux + (long)i * r8)[lane] = t < p.V ? __ldg(reinterpret_cast<const uint4*>(u) + lane) : zero;
            } else {
                for (int k = lane; k < r8; k += 32) {
                    float x[3];
                    bf16_parts(t < p.V && k < p.r ? load_one(u + k) : 0.0f, x);
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        if (q < planes) put<bf16_t>(b.ux, ((long)q * n + i) * r8 + k, x[q]);
                }
            }
        }
        return;
    }
    const int i = blockIdx.x * kMarkovWarps + warp;
    const int mine = i < n ? token_of(i, &bad) : 0;
    if (bad && lane == 0) atomicOr(b.status, SPEC_DEV_TOKEN);
    int less = 0, same = 0, before = 0;   // tokens below this one, rows of it, those of them before this one
    for (int lo = 0; lo < n; lo += kOrderTile) {
        __syncthreads();
#pragma unroll
        for (int k = threadIdx.x; k < kOrderTile; k += kMarkovThreads)
            if (lo + k < n) s_tok[k] = token_of(lo + k, &bad);
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
}

// A few rows: one pass over the vocabulary forms both products.  A warp takes an entry v, its lanes
// the r columns: dWt[v] = sum_i dz[i, v] U[x_i] with the rows' U in registers, and dX's sums, one per row
// and column, in registers too.  Bound by memory: Wt in, dWt and dU's zeros out.  7 rows, V = 248,320,
// r = 256: the tensor cores would spend their steps of 64 rows on zeros.
template <typename G, typename W, int C>
__global__ void __launch_bounds__(kMarkovThreads) markov_small_kernel(MarkovParams p, MarkovBind b) {
    constexpr int N = kMarkovSmall, kV = 64;       // entries of a turn
    __shared__ __align__(16) float s_d[kV][N];
    __shared__ float s_x[kMarkovWarps][32 * C];
    __shared__ int s_row[N];
    const int n = p.B * p.gamma, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < N) s_row[tid] = p.V;
    __syncthreads();
    if (tid < n) s_row[b.order[tid]] = b.token[tid];
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
// they are all, that is dU's row, otherwise the sum is kept for markov_runs_kernel.  Terms are (row, part) in
// order; 16-byte columns go over lanes and the terms over groups of threads, whose sums meet in order.
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
__global__ void __launch_bounds__(kJoinThreads) markov_join_kernel(MarkovParams p, MarkovBind b, MarkovJoin a) {
    __shared__ float4 s_sum[kJoinThreads];
    const int at = blockIdx.x, t = b.token[at];
    const int2 run = b.run[at];
    if (t >= p.V || (at - run.x) % kJoinRun != 0) return;
    const int rows = min(kJoinRun, run.x + run.y - at);
    const int quads = round4(p.r) / 4, groups = kJoinThreads / quads;
    const int k = threadIdx.x % quads, g = threadIdx.x / quads, terms = rows * a.parts;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (g < groups) {
        const int lo = terms * g / groups, hi = terms * (g + 1) / groups;
#pragma unroll 8
        for (int e = lo; e < hi; ++e) {
            const int q = e / a.parts, part = e - q * a.parts, i = b.order[at + q];
            const float4 x = *reinterpret_cast<const float4*>(b.part + (part * a.part_stride + i) * a.pitch + 4 * k);
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
    }
    if (!join_meet(s_sum, s, k, g, quads, groups)) return;
    if (run.y <= kJoinRun) join_out(p, t, k, s);
    else reinterpret_cast<float4*>(b.runs + (long)at * round4(p.r))[k] = s;
}
// The tokens of more rows: a CTA looks at 32 places for where one begins.
__global__ void __launch_bounds__(kJoinThreads) markov_runs_kernel(MarkovParams p, MarkovBind b) {
    __shared__ float4 s_sum[kJoinThreads];
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

static bool markov_small(int n) { return n <= kMarkovSmall; }

static size_t markov_bind(MarkovBind& b, void* ws, int n, int r, int V) {
    uint8_t* w = reinterpret_cast<uint8_t*>(ws);
    b.status = &reinterpret_cast<WsHeader*>(ws)->status;
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
    if (markov_small(n)) {
        b.part = reinterpret_cast<float*>(take((size_t)kMarkovSlabs * n * round4(r) * 4));
        return at;
    }
    const int columns = markov_slice(n, r, V);
    b.none = reinterpret_cast<unsigned long long*>(take((size_t)(n + 63) / 64 * 8));
    b.ux = reinterpret_cast<bf16_t*>(take((size_t)3 * n * round8(r) * 2));
    const MarkovTc whole = markov_tc_dx(n, V), part = markov_tc_dx(n, columns);
    const size_t parts = whole.parts > part.parts ? whole.parts : part.parts;
    b.part = reinterpret_cast<float*>(take(parts * whole.tiles * 256 * (r > 128 ? 256 : 128) * 4));
    b.zs = reinterpret_cast<bf16_t*>(take((size_t)3 * n * round8(columns) * 2));
    b.ws = reinterpret_cast<bf16_t*>(take((size_t)3 * columns * round8(r) * 2));
    return at;
}

size_t markov_grad_workspace_bytes(int B, int gamma, int V, int r) {
    MarkovBind b;
    return markov_bind(b, nullptr, B * gamma, r, V);
}

template <typename G, typename W>
static int markov_small_launch(const MarkovParams& p, const MarkovBind& b, cudaStream_t stream) {
    int slabs = (p.V + 63) / 64;
    const int most = 2 * device_sm_count() < kMarkovSlabs ? 2 * device_sm_count() : kMarkovSlabs;
    if (slabs > most) slabs = most;
    const int C = (p.r + 31) / 32;
    if (C <= 1) markov_small_kernel<G, W, 1><<<slabs, kMarkovThreads, 0, stream>>>(p, b);
    else if (C <= 2) markov_small_kernel<G, W, 2><<<slabs, kMarkovThreads, 0, stream>>>(p, b);
    else if (C <= 4) markov_small_kernel<G, W, 4><<<slabs, kMarkovThreads, 0, stream>>>(p, b);
    else markov_small_kernel<G, W, 8><<<slabs, kMarkovThreads, 0, stream>>>(p, b);
    return slabs;
}

cudaError_t markov_grad_launch(const MarkovParams& p, void* ws, cudaStream_t stream) {
    const int n = p.B * p.gamma;
    MarkovBind b;
    markov_bind(b, ws, n, p.r, p.V);
    const bool small = markov_small(n), g16 = p.gdt == SPEC_BF16, w16 = p.wdt == SPEC_BF16;
    const unsigned grid = (n + kMarkovWarps - 1) / kMarkovWarps + (small ? 0 : (n + 63) / 64);
    if (w16) markov_order_kernel<bf16_t><<<grid, kMarkovThreads, 0, stream>>>(p, b, 1);
    else markov_order_kernel<float><<<grid, kMarkovThreads, 0, stream>>>(p, b, 3);
    MarkovJoin join = {0, n, round4(p.r)};
    if (small) {
        join.parts = g16 ? (w16 ? markov_small_launch<bf16_t, bf16_t>(p, b, stream) : markov_small_launch<bf16_t, float>(p, b, stream))
                         : (w16 ? markov_small_launch<float, bf16_t>(p, b, stream) : markov_small_launch<float, float>(p, b, stream));
    } else {
        const cudaError_t e = markov_tc_launch(p, b, &join, stream);
        if (e != cudaSuccess) return e;
    }
    markov_join_kernel<<<n, kJoinThreads, 0, stream>>>(p, b, join);
    if (n > kJoinRun) markov_runs_kernel<<<(n + 31) / 32, kJoinThreads, 0, stream>>>(p, b);
    return cudaGetLastError();
}

}  // namespace spec
