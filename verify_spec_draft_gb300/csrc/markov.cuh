// markov.cuh - what the kernels of spec_markov_grad share (markov.cu, markov_tc.cu).
#pragma once

#include "internal.h"
#include "row_words.cuh"

namespace spec {

constexpr int kMarkovPairs = 76;                 // most CTA pairs of a tensor-core product

struct MarkovBind {
    unsigned* status;
    int32_t* order;          // [n] the rows by (token, row); rows without a token behind all others
    int32_t* token;          // [n] their tokens in that order (V: none)
    int32_t* of_row;         // [n] the rows' tokens (V: none)
    unsigned long long* none;   // [ceil(n / 64)] rows without a token, a bit each
    bf16_t* ux;              // [n, r] U[x_i], 0 for a row without a token (tensor cores)
    float* dx;               // dX in parts: [parts][n][r], or the pairs' tiles
    int parts;
};

// A tensor-core product's items: tiles of 256 outputs over `steps` steps each, dealt to pairs.
struct MarkovTc { int tiles, steps, pairs; };
// The contraction over the vocabulary has few tiles, so all their steps in a line are cut into equal
// shares: pair q has steps [mtc_begin(q), mtc_begin(q + 1)), and its part of a tile is kept at place
// q + tile.
__host__ __device__ inline long mtc_begin(const MarkovTc& a, int q) { return (long)a.tiles * a.steps * q / a.pairs; }
__host__ __device__ inline int mtc_pair_of(const MarkovTc& a, long step) {   // the pair whose share step is in
    const long all = (long)a.tiles * a.steps;
    int q = (int)((step * a.pairs + a.pairs - 1) / all);
    if (q > a.pairs - 1) q = a.pairs - 1;
    while (q > 0 && mtc_begin(a, q) > step) --q;
    while (q + 1 < a.pairs && mtc_begin(a, q + 1) <= step) ++q;
    return q;
}

template <typename T> __device__ __forceinline__ void put(void* o, long i, float x);
template <> __device__ __forceinline__ void put<float>(void* o, long i, float x) { reinterpret_cast<float*>(o)[i] = x; }
template <> __device__ __forceinline__ void put<bf16_t>(void* o, long i, float x) {
    reinterpret_cast<unsigned short*>(o)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
__device__ __forceinline__ void put(void* o, int dtype, long i, float x) {
    if (dtype == SPEC_BF16) put<bf16_t>(o, i, x);
    else put<float>(o, i, x);
}

bool markov_tc_supported(const MarkovParams& p);
cudaError_t markov_tc_launch(const MarkovParams& p, const MarkovBind& b, cudaStream_t stream);

}  // namespace spec
