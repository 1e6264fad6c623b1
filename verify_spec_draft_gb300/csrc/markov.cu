// markov.cu - the gradients of the Markov bias weights (spec_markov_grad).
//
// The biased rows are z_i = l_i + Wt U[x_i] (x_i the token before position i), so with dz the
// rows' gradient and n = B gamma rows
//     dWt = dz^T Ux          [V, r], Ux the gathered rows U[x_i]       contraction over n
//     dX  = dz Wt            [n, r]                                    contraction over V
//     dU[x] = the sum of dX's rows with x_i = x, in the rows' order
// Four steps on the stream: the rows' tokens in order, with Ux beside them; dWt; dX in parts of
// the vocabulary; and dU, which joins the parts of each token's rows.
#include "markov.cuh"

namespace spec {

constexpr int kMarkovTile = 64;                  // outputs of a tile's side
constexpr int kMarkovStep = 16;                  // terms of a contraction step
constexpr int kMarkovThreads = 256;
constexpr int kMarkovMaxParts = 256;

// Parts of the vocabulary that dX is summed in: as many as fill the device.
static int markov_parts(int n, int r, int V, int sms) {
    const int tiles = ((n + kMarkovTile - 1) / kMarkovTile) * ((r + kMarkovTile - 1) / kMarkovTile);
    int parts = (4 * sms + tiles - 1) / tiles;
    const int most = (V + 127) / 128;
    if (parts > most) parts = most;
    return parts < 1 ? 1 : (parts > kMarkovMaxParts ? kMarkovMaxParts : parts);
}

constexpr int kOrderTile = 2048;                 // tokens compared at a time

// Row i's place among the rows by (token, row), counted: n comparisons a row, a warp a row.  With
// `gather` a second half of the grid copies the rows U[x_i] and marks the rows without a token.
__global__ void __launch_bounds__(kMarkovThreads) markov_order_kernel(MarkovParams p, MarkovBind b, bool gather) {
    __shared__ int32_t s_tok[kOrderTile];
    const int n = p.B * p.gamma, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto token_of = [&](int i, bool* bad) {
        const int q = i / p.gamma, j = i - q * p.gamma;
        const int t = j == 0 ? p.anchor[q] : p.tokens[(long)q * p.gamma + j - 1];
        if (t < -1 || t >= p.V) *bad = true;
        return t < 0 || t >= p.V ? p.V : t;
    };
    bool bad = false;
    const int rows = kMarkovThreads / 32, ranks = (n + rows - 1) / rows;
    if ((int)blockIdx.x >= ranks) {   // (a CTA of 64 rows, so that it has a whole word of marks)
        const int i0 = ((int)blockIdx.x - ranks) * 64;
        if (warp == 0) {
            const unsigned lo = __ballot_sync(0xffffffffu, i0 + lane < n && token_of(i0 + lane, &bad) >= p.V);
            const unsigned hi = __ballot_sync(0xffffffffu, i0 + 32 + lane < n && token_of(i0 + 32 + lane, &bad) >= p.V);
            if (lane == 0) b.none[i0 >> 6] = (unsigned long long)hi << 32 | lo;
        }
        for (int i = i0 + warp; i < min(n, i0 + 64); i += rows) {
            const int t = token_of(i, &bad);
            const uint4* u = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16_t*>(p.U) + (long)t * p.r);
            uint4* o = reinterpret_cast<uint4*>(b.ux + (long)i * p.r);
            if (lane < p.r / 8) o[lane] = t < p.V ? __ldg(u + lane) : make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int i = blockIdx.x * rows + warp;
    const int mine = i < n ? token_of(i, &bad) : 0;
    if (bad && lane == 0) atomicOr(b.status, SPEC_DEV_TOKEN);
    int rank = 0;
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
            rank += t < mine || (t == mine && lo + k < i) ? 1 : 0;
        }
    }
    rank = (int)__reduce_add_sync(0xffffffffu, (unsigned)rank);
    if (i < n && lane == 0) {
        b.order[rank] = i;
        b.token[rank] = mine;
        b.of_row[i] = mine;
    }
}
static void markov_order(const MarkovParams& p, const MarkovBind& b, bool gather, cudaStream_t stream) {
    const int n = p.B * p.gamma, rows = kMarkovThreads / 32;
    markov_order_kernel<<<(n + rows - 1) / rows + (gather ? (n + 63) / 64 : 0), kMarkovThreads, 0, stream>>>(p, b, gather);
}

// A 64 x 64 tile of sums on CUDA cores, 4 x 4 outputs a thread: s_a[step][a], s_b[step][b].
__device__ __forceinline__ void tile_step(const float (*s_a)[kMarkovTile + 4], const float (*s_b)[kMarkovTile + 4],
                                          float (&acc)[4][4], int ty, int tx) {
#pragma unroll
    for (int k = 0; k < kMarkovStep; ++k) {
        const float4 a = *reinterpret_cast<const float4*>(&s_a[k][ty * 4]), b = *reinterpret_cast<const float4*>(&s_b[k][tx * 4]);
        const float x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int w = 0; w < 4; ++w) acc[h][w] = fmaf(x[h], y[w], acc[h][w]);
    }
}

// dWt's tile [64 entries, 64 k], and dU's rows of those entries set to 0.
template <typename G, typename W>
__global__ void __launch_bounds__(kMarkovThreads) markov_wt_kernel(MarkovParams p, MarkovBind b) {
    __shared__ __align__(16) float s_a[kMarkovStep][kMarkovTile + 4], s_b[kMarkovStep][kMarkovTile + 4];
    const int n = p.B * p.gamma, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int v0 = blockIdx.x * kMarkovTile, k0 = blockIdx.y * kMarkovTile;
    const G* dz = reinterpret_cast<const G*>(p.grad);
    const W* U = reinterpret_cast<const W*>(p.U);
    float acc[4][4] = {};
    for (int i0 = 0; i0 < n; i0 += kMarkovStep) {
        __syncthreads();
        for (int e = tid; e < kMarkovStep * kMarkovTile; e += kMarkovThreads) {
            const int i = i0 + e / kMarkovTile, c = e % kMarkovTile;
            const int t = i < n ? b.of_row[i] : p.V;
            const bool on = t < p.V;
            s_a[e / kMarkovTile][c] = on && v0 + c < p.V ? load_one(dz + (long)i * p.ld + v0 + c) : 0.0f;
            s_b[e / kMarkovTile][c] = on && k0 + c < p.r ? load_one(U + (long)t * p.r + k0 + c) : 0.0f;
        }
        __syncthreads();
        tile_step(s_a, s_b, acc, ty, tx);
    }
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int v = v0 + ty * 4 + h, k = k0 + tx * 4 + w;
            if (v >= p.V || k >= p.r) continue;
            put(p.dWt_out, p.odt, (long)v * p.r + k, acc[h][w]);
            put(p.dU_out, p.odt, (long)v * p.r + k, 0.0f);
        }
}

// dX's tile [64 rows, 64 k] over one part of the vocabulary.
template <typename G, typename W>
__global__ void __launch_bounds__(kMarkovThreads) markov_dx_kernel(MarkovParams p, MarkovBind b) {
    __shared__ __align__(16) float s_a[kMarkovStep][kMarkovTile + 4], s_b[kMarkovStep][kMarkovTile + 4];
    const int n = p.B * p.gamma, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int i0 = blockIdx.x * kMarkovTile, k0 = blockIdx.y * kMarkovTile, part = blockIdx.z;
    const int lo = (int)((long)p.V * part / b.parts), hi = (int)((long)p.V * (part + 1) / b.parts);
    const G* dz = reinterpret_cast<const G*>(p.grad);
    const W* Wt = reinterpret_cast<const W*>(p.Wt);
    float acc[4][4] = {};
    for (int v0 = lo; v0 < hi; v0 += kMarkovStep) {
        __syncthreads();
        for (int e = tid; e < kMarkovStep * kMarkovTile; e += kMarkovThreads) {
            const int a = e % kMarkovStep, i = i0 + e / kMarkovStep, v = v0 + a;
            s_a[a][e / kMarkovStep] = i < n && v < hi && b.of_row[i] < p.V ? load_one(dz + (long)i * p.ld + v) : 0.0f;
            const int c = e % kMarkovTile, u = v0 + e / kMarkovTile;
            s_b[e / kMarkovTile][c] = u < hi && k0 + c < p.r ? load_one(Wt + (long)u * p.r + k0 + c) : 0.0f;
        }
        __syncthreads();
        tile_step(s_a, s_b, acc, ty, tx);
    }
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int i = i0 + ty * 4 + h, k = k0 + tx * 4 + w;
            if (i < n && k < markov_pitch(p.r)) b.dx[((long)part * n + i) * markov_pitch(p.r) + k] = acc[h][w];
        }
}

// dU's rows: the CTA at a token's first place among the ordered rows joins that token's.  Its terms
// are (row, part) in order; 16-byte columns go over lanes and the terms over groups of threads, whose
// sums meet in order.
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) markov_join_kernel(MarkovParams p, MarkovBind b, MarkovJoin a) {
    __shared__ float4 s_sum[kJoinThreads];
    const int n = p.B * p.gamma, at = blockIdx.x;
    const int t = b.token[at];
    if (t >= p.V || (at > 0 && b.token[at - 1] == t)) return;
    int end = n;   // the last row of this token, found by halves: tokens are in order
    for (int lo = at + 1; lo < end;) {
        const int mid = (lo + end) >> 1;
        if (b.token[mid] == t) lo = mid + 1; else end = mid;
    }
    const int quads = (p.r + 3) / 4, groups = kJoinThreads / quads;
    const int k = threadIdx.x % quads, g = threadIdx.x / quads;
    const int terms = (end - at) * a.parts;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (g < groups) {
        const int lo = (int)((long)terms * g / groups), hi = (int)((long)terms * (g + 1) / groups);
#pragma unroll 8
        for (int e = lo; e < hi; ++e) {
            const int q = e / a.parts, part = e - q * a.parts, i = b.order[at + q];
            const float4 x = *reinterpret_cast<const float4*>(b.dx + (part * a.part_stride + i) * a.pitch + 4 * k);
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
        s_sum[g * quads + k] = s;
    }
    __syncthreads();
    if (g != 0) return;
    for (int q = 1; q < groups; ++q) {
        const float4 x = s_sum[q * quads + k];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    const float o[4] = {s.x, s.y, s.z, s.w};
    for (int h = 0; h < 4 && 4 * k + h < p.r; ++h) put(p.dU_out, p.odt, (long)t * p.r + 4 * k + h, o[h]);
}
void markov_join(const MarkovParams& p, const MarkovBind& b, const MarkovJoin& a, cudaStream_t stream) {
    markov_join_kernel<<<p.B * p.gamma, kJoinThreads, 0, stream>>>(p, b, a);
}

static size_t markov_bind(MarkovBind& b, void* ws, int n, int r, int V) {
    uint8_t* w = reinterpret_cast<uint8_t*>(ws);
    b.status = &reinterpret_cast<WsHeader*>(ws)->status;
    size_t at = kWsHeaderBytes;
    b.order = reinterpret_cast<int32_t*>(w + at);
    at += align256((size_t)n * 4);
    b.token = reinterpret_cast<int32_t*>(w + at);
    at += align256((size_t)n * 4);
    b.of_row = reinterpret_cast<int32_t*>(w + at);
    at += align256((size_t)n * 4);
    b.none = reinterpret_cast<unsigned long long*>(w + at);
    at += align256((size_t)(n + 63) / 64 * 8);
    b.ux = reinterpret_cast<bf16_t*>(w + at);
    at += align256((size_t)n * r * 2);
    b.dx = reinterpret_cast<float*>(w + at);
    const size_t plain = (size_t)b.parts * n * markov_pitch(r) * 4;
    const MarkovTc dx = markov_tc_dx(n, V);
    const size_t tiles = (size_t)dx.tiles * dx.parts * 256 * (r > 128 ? 256 : 128) * 4;
    at += align256(plain > tiles ? plain : tiles);
    return at;
}

size_t markov_grad_workspace_bytes(int B, int gamma, int V, int r) {
    MarkovBind b;
    b.parts = markov_parts(B * gamma, r, V, 152);
    return markov_bind(b, nullptr, B * gamma, r, V);
}

template <typename G, typename W>
static void markov_typed(const MarkovParams& p, const MarkovBind& b, cudaStream_t stream) {
    const int n = p.B * p.gamma;
    auto tiles = [](int x) { return (unsigned)((x + kMarkovTile - 1) / kMarkovTile); };
    markov_wt_kernel<G, W><<<dim3(tiles(p.V), tiles(p.r)), kMarkovThreads, 0, stream>>>(p, b);
    markov_dx_kernel<G, W><<<dim3(tiles(n), tiles(p.r), (unsigned)b.parts), kMarkovThreads, 0, stream>>>(p, b);
}

cudaError_t markov_grad_launch(const MarkovParams& p, void* ws, cudaStream_t stream) {
    const int n = p.B * p.gamma;
    MarkovBind b;
    b.parts = markov_parts(n, p.r, p.V, 152);
    markov_bind(b, ws, n, p.r, p.V);
    const bool tc = markov_tc_supported(p);
    markov_order(p, b, tc, stream);
    if (tc) return markov_tc_launch(p, b, stream);
    const bool g16 = p.gdt == SPEC_BF16, w16 = p.wdt == SPEC_BF16;
    if (g16 && w16) markov_typed<bf16_t, bf16_t>(p, b, stream);
    else if (g16) markov_typed<bf16_t, float>(p, b, stream);
    else if (w16) markov_typed<float, bf16_t>(p, b, stream);
    else markov_typed<float, float>(p, b, stream);
    markov_join(p, b, {b.parts, n, markov_pitch(p.r)}, stream);
    return cudaGetLastError();
}

}  // namespace spec
