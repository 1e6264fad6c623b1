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

// A tensor-core product's items: tiles of 256 outputs, each in `parts` ranges of its steps.  Item
// i is part i / tiles of tile i % tiles, and the pairs take them in order, so the tiles that
// run at the same time go through the same steps and read B's rows from memory once.
struct MarkovTc { int tiles, steps, parts; };
__host__ __device__ inline int mtc_begin(const MarkovTc& a, int part) { return (int)((long)a.steps * part / a.parts); }

template <typename T> __device__ __forceinline__ void put(void* o, long i, float x);
template <> __device__ __forceinline__ void put<float>(void* o, long i, float x) { reinterpret_cast<float*>(o)[i] = x; }
template <> __device__ __forceinline__ void put<bf16_t>(void* o, long i, float x) {
    reinterpret_cast<unsigned short*>(o)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
__device__ __forceinline__ void put(void* o, int dtype, long i, float x) {
    if (dtype == SPEC_BF16) put<bf16_t>(o, i, x);
    else put<float>(o, i, x);
}

// Where the join finds row i's part: dx[(part * part_stride + i) * pitch], 16 bytes aligned.
struct MarkovJoin { int parts; long part_stride; int pitch; };
__host__ __device__ inline int markov_pitch(int r) { return (r + 3) & ~3; }
void markov_join(const MarkovParams& p, const MarkovBind& b, const MarkovJoin& a, cudaStream_t stream);

MarkovTc markov_tc_dx(int n, int V);
bool markov_tc_supported(const MarkovParams& p);
cudaError_t markov_tc_launch(const MarkovParams& p, const MarkovBind& b, cudaStream_t stream);

}  // namespace spec
