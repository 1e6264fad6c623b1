// markov.cuh - what the kernels of spec_markov_grad share (markov.cu, markov_tc.cu).
#pragma once

#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kMarkovPairs = 76;                 // CTA pairs that a tensor-core product is cut for
constexpr int kMarkovSmall = 8;                  // rows that one pass over the weights takes
constexpr int kMarkovSlabs = 304;                // most slabs of that pass
constexpr int kJoinRun = 8;                      // rows of a token that one CTA joins
constexpr size_t kMarkovStage = 96u << 20;       // bytes that are staged at a time, about

struct MarkovBind {
    unsigned* status;
    int32_t* order;          // [n] the rows by (token, row); rows without a token behind all others
    int32_t* token;          // [n] their tokens in that order (V: none)
    int2* run;               // [n] there: where the token's rows begin, and how many they are
    uint8_t* none;           // [ceil(n / 64) * 8] rows without a token, a bit each
    unsigned* unclean;       // whether one holds what is not finite (returned to 0 by markov_runs_kernel)
    bf16_t* ux;              // [planes][n][r8] U[x_i], 0 for a row without a token
    float* part;             // dX in parts
    float* runs;             // [n][r4] sums over kJoinRun rows of a token
    bf16_t* stage;           // slices of dz [planes][n][columns] and Wt [planes][columns][r8]
    size_t stage_bytes;
};

__host__ __device__ inline int round8(int r) { return (r + 7) & ~7; }
__host__ __device__ inline int round4(int r) { return (r + 3) & ~3; }

// A tensor-core product's items: tiles of 256 outputs, each in `parts` parts of its steps.  Item i is
// part i / tiles of tile i % tiles, and the product's pairs take them in order.  A part takes every
// parts-th block of `block` steps, so that all pairs go along the contraction together: what one has
// read from memory the others find in L2.  With operands in several planes (float32 values as
// sums of bf16) a part's steps run through the pairs of planes.
struct MarkovTc {
    int tiles, steps, parts, block;
    int first, pairs;        // its CTA pairs
    int terms;               // pairs of planes
    unsigned planes;         // their numbers, 2 bits for A and 2 for B each, from the lowest
    int v0, v1;              // the entries that this launch covers
    int add;                 // parts are added to what is there
};
constexpr int kMarkovItems = 2 * kMarkovPairs;   // most parts of dX in all, where there are fewer tiles

template <typename T> __device__ __forceinline__ void put(void* o, long i, float x);
template <> __device__ __forceinline__ void put<float>(void* o, long i, float x) { reinterpret_cast<float*>(o)[i] = x; }
template <> __device__ __forceinline__ void put<bf16_t>(void* o, long i, float x) {
    reinterpret_cast<unsigned short*>(o)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
__device__ __forceinline__ void put(void* o, int dtype, long i, float x) {
    if (dtype == SPEC_BF16) put<bf16_t>(o, i, x);
    else put<float>(o, i, x);
}

// A float32 value as a sum of bf16 ones, 24 bits in three; what is not finite stays in the first.
__device__ __forceinline__ float bf16_part(float x) {
    const float a = __bfloat162float(__float2bfloat16_rn(x));
    return fabsf(a) < INFINITY || !(fabsf(x) < INFINITY) ? a : __bfloat162float(__float2bfloat16_rz(x));
}
__device__ __forceinline__ void bf16_parts(float x, float (&o)[3]) {
    o[0] = bf16_part(x);
    const float r = fabsf(o[0]) < INFINITY ? x - o[0] : 0.0f;
    o[1] = bf16_part(r);
    o[2] = bf16_part(r - o[1]);
}

// A kernel launched as the programmatic dependent of the one before it: it is set up meanwhile, and waits for
// that one before it reads or writes anything but the call's inputs.
template <typename... P, typename... A>
inline cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Where the join finds row i's part: part[(p * part_stride + i) * pitch], 16 bytes aligned.
struct MarkovJoin { int parts; long part_stride; int pitch; };

// The entries of a staged slice: about kMarkovStage bytes of three planes of dz and Wt.
__host__ inline int markov_slice(int n, int r, int V) {
    const size_t most = kMarkovStage / ((size_t)(n + round8(r)) * 6) / 256 * 256;
    return most < 256 ? 256 : (most < (size_t)V ? (int)most : V);
}
cudaError_t markov_join(const MarkovParams& p, const MarkovBind& b, const MarkovJoin& a, cudaStream_t stream);
// both products and the join of dX's parts
cudaError_t markov_tc_launch(const MarkovParams& p, const MarkovBind& b, cudaStream_t stream);

}  // namespace spec
