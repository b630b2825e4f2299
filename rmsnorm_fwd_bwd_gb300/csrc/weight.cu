// weight.cu -- a weight matrix [N, K] as e4m3 codes with one scale per block of 128 x 128.
//
// scale = max(max|w| / 448, 2^-126) of the block (pow2: up to the next power of two), code =
// w / scale rounded to nearest-even, both quotients exactly rounded: the same codes wherever
// a checkpoint is turned into them. A block of 256 threads holds one block of the weight in
// registers (eight octets a thread), so that the weight is read once. Bound by HBM: the
// weight in, a byte per entry out.
#include "octet.cuh"
#include "quant.cuh"
#include "serving.h"

namespace rmsnorm {
namespace {

constexpr int kThreads = 256;
constexpr int kOctets = 128 * 128 / 8 / kThreads;  // per thread

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) quant_weight_blocks(const WeightArgs a) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    __shared__ float part[kThreads / 32];
    const int o = threadIdx.x & 15;  // the octet's column in the block; 16 threads hold a row
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / a.kblocks) * 128 + (threadIdx.x >> 4);
    const int kb = static_cast<int>(blockIdx.x % a.kblocks);
    const int col = kb * 128 + o * 8;
    const int width = min(max(a.K - col, 0), 8);
    griddep_wait();
    const char* w = static_cast<const char*>(a.w) + (row0 * a.ldw + col) * EB;
    uint32_t v[kOctets][W];
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
        const int hi = row0 + 16 * i < a.N ? width : 0;
#pragma unroll
        for (int j = 0; j < W; ++j) v[i][j] = 0u;
        if (hi > 0) octet_load<DT, ALIGNED>(w + i * 16 * a.ldw * EB, 0, hi, v[i]);
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
        uint64_t z[4];
        octet_pairs<DT>(v[i], z);
        amax = max_magnitude(amax, octet_amax<true>(z, 0, 8));
    }
    amax = warp_allmax(amax);
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = warp_allmax(part[lane & (kThreads / 32 - 1)]);
    float s = amax / 448.0f;
    if (s < 1.17549435e-38f) s = 1.17549435e-38f;  // 2^-126; a NaN stays
    if (a.pow2) s = power_of_two_above(s);
    if (threadIdx.x == 0) a.scales[static_cast<int64_t>(blockIdx.x / a.kblocks) * a.ldscales + kb] = s;
    const bool first = o == 0, last = o == 15 || col + 8 >= a.K;
    char* out = static_cast<char*>(a.codes) + row0 * a.ldcodes + col;
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
        float f[8];
        Oct<DT>::unpack(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] /= s;
        uint32_t code[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            code[j] = e4m3_pair(f2_pack(f[4 * j], f[4 * j + 1]), 1.f) | e4m3_pair(f2_pack(f[4 * j + 2], f[4 * j + 3]), 1.f) << 16;
        octet_store<1, 2, ALIGNED>(out + i * 16 * a.ldcodes, code, row0 + 16 * i < a.N ? width : 0, first, last);
    }
    griddep_launch_dependents();
}

}  // namespace

const void* weight_kernel(int dtype, bool aligned) {
    switch (dtype) {
    case kF32: return aligned ? reinterpret_cast<const void*>(&quant_weight_blocks<kF32, true>)
                              : reinterpret_cast<const void*>(&quant_weight_blocks<kF32, false>);
    case kF16: return aligned ? reinterpret_cast<const void*>(&quant_weight_blocks<kF16, true>)
                              : reinterpret_cast<const void*>(&quant_weight_blocks<kF16, false>);
    case kBF16: return aligned ? reinterpret_cast<const void*>(&quant_weight_blocks<kBF16, true>)
                               : reinterpret_cast<const void*>(&quant_weight_blocks<kBF16, false>);
    default: return nullptr;
    }
}

int weight_threads() { return kThreads; }

}  // namespace rmsnorm
