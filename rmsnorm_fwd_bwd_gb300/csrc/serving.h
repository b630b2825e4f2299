// serving.h -- host-side interface between the entry points of
// include/rmsnorm_serving.h (serving_api.cu) and their kernels (matmul.cu, weight.cu,
// append.cu). Internal: not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fused.h"

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
    int wide_bias;     // there is a bias, and it starts on one
    uint32_t* err;     // device error word
    int give_up;       // debug builds: block of each cluster that acts as if a wait had given up, or -1
};

// Most blocks that share K: the portable size of a cluster.
constexpr int kMatmulMostSplit = 8;

// Tiles of a product: 256 rows of a by 256 of b, of a pair of blocks; 128 by 128; or 128 rows of
// b by `n` rows of a, with K split over the blocks of a cluster.
enum MatmulTiles { kMatmulPair = 0, kMatmulWide, kMatmulThin };

struct MatmulPlan {
    int dtype = 0;
    MatmulTiles how = kMatmulPair;
    bool tma = false;  // tiles by TMA, which wants a's and b's rows on 16-byte boundaries
    int n = 0;         // thin: rows of a
    int cluster = 1;   // blocks
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

// Heads of one kind of an append: queries (y: their output, y_token a token's stride), keys or
// values (y: the cache's rows, y_token the stride between a page's rows).
struct AppendSet : RopeSet {
    int64_t y_page;
    float* scales;  // of e4m3 rows; null: rows in the heads' type
    int64_t scale_page, scale_row, scale_head;
};

// The rotation's members are RopeArgs' (its sets are not used); a kind that is missing has no
// heads.
struct AppendArgs : RopeArgs {
    AppendSet sets[3];
    int first[3];              // block with which a kind starts
    const int64_t* slots;
    int64_t pages;
    int page_size;
    uint32_t* err;
};

const void* append_kernel(const RopePlan& p, bool codes);

const void* matmul_kernel(const MatmulPlan& p);
// Threads and shared memory of a plan whose other members are set.
void matmul_shape(MatmulPlan& p);

}  // namespace rmsnorm
