// serving.h -- host-side interface between the entry points of
// include/rmsnorm_serving.h (serving_api.cu) and their kernels (matmul.cu, weight.cu,
// append.cu). Internal: not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsnorm {

// The 8-bit product y = (a sa) (b sb)^T + bias.
struct MatmulArgs {
    const uint8_t* a;
    const float* sa;
    const uint8_t* b;
    const float* sb;
    const void* bias;  // may be null
    void* y;
    int64_t lda, ldsa, ldb, ldsb, ldy;
    int64_t M;
    int N, K;
    int kblocks;       // of 128 codes
    int per_row;       // one scale per row of a
    int m_tiles, n_tiles;
    int wide_y;        // y's rows on 16-byte boundaries
    uint32_t* err;     // device error word
};

// A launch shape. wide: tiles of 128 rows of a by 128 or 256 of b (`n`), persistent blocks;
// else tiles of 128 rows of b by `n` rows of a, K split over clusters of `split` blocks.
struct MatmulPlan {
    int dtype = 0;
    bool wide = false;
    bool tma = false;  // tiles by TMA, which wants a's and b's rows on 16-byte boundaries
    int n = 0;
    int split = 1;
    int threads = 0;
    int64_t blocks = 0;
    size_t smem = 0;
};

// A weight [N, K] as codes with scales per block of 128 x 128.
struct WeightArgs {
    const void* w;
    void* codes;
    float* scales;
    int64_t ldw, ldcodes, ldscales;
    int N, K, kblocks;
    int pow2;
};

const void* weight_kernel(int dtype, bool aligned);
int weight_threads();

const void* matmul_kernel(const MatmulPlan& p);
// Threads and shared memory of a plan whose other members are set.
void matmul_shape(MatmulPlan& p);

}  // namespace rmsnorm
