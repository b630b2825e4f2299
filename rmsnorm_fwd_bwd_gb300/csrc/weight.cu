// weight.cu -- a weight matrix [N, K] as e4m3 codes with one scale per block of 128 x 128.
//
// scale = max(max|w| / 448, 2^-126) of the block (pow2: up to the next power of two), code =
// w / scale rounded to nearest-even, both quotients exactly rounded: the same codes wherever
// a checkpoint is turned into them. A block of 512 threads holds one block of the weight in
// registers (four octets a thread), so that the weight is read once. Bound by the blocks' phases,
// loads, maximum, stores, three blocks to an SM: 8192 x 8192 bf16 40.6 us (5.0 TB/s; 46.6 with two
// blocks, 54 with persistent ones that load ahead), 4099 x 5000 fp32 17.8 (5.8 TB/s). Rows off 16 bytes,
// whose words are shifted together: 8192 x 8191 bf16 76.5 us (2.6 TB/s), 4099 x 4999 fp32 32.7 (3.1). Three
// blocks leave 40 registers a thread: fp32 spills 44 bytes, off 16 bytes 152 of them.
#include "octet.cuh"
#include "quant.cuh"
#include "serving.h"

namespace rmsnorm {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = kThreads / 16;                // of a block at a time: 16 threads hold a row
constexpr int kOctets = 128 / kRows;                // per thread

// The largest magnitude among a thread's words, as bits: those of numbers without their sign are in
// the numbers' order, infinity above them and NaN above that. 16-bit types: two to a word.
template <int DT> __device__ __forceinline__ uint32_t larger_bits(uint32_t m, uint32_t w) {
    return DT == kF32 ? max(m, w & 0x7fffffffu) : __vmaxu2(m, w & 0x7fff7fffu);
}
template <int DT> __device__ __forceinline__ float bits_value(uint32_t m) {
    if (DT == kF32) return __uint_as_float(m);
    const uint32_t v = max(m >> 16, m & 0xffffu);
    return DT == kF16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(v))) : __uint_as_float(v << 16);
}

// Codes of w / s for an octet. w times the inverse of s is off by less than 2^-22 of the quotient, the
// inverse's rounding included: where the codes of w times a little less (`less`) and a little more
// are one, it is the quotient's; else, near the border between two, the quotients are taken
// (about one octet in 10^4; with quotients throughout 8192 x 8192 bf16 took 62.5 us).
template <int DT>
__device__ __forceinline__ void octet_quotients(const uint32_t (&w)[Oct<DT>::kWords], float s, float less, float more,
                                                uint32_t (&code)[2]) {
    uint64_t z[4];
    octet_pairs<DT>(w, z);
    uint32_t other[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        code[i] = e4m3_pair(z[2 * i], less) | e4m3_pair(z[2 * i + 1], less) << 16;
        other[i] = e4m3_pair(z[2 * i], more) | e4m3_pair(z[2 * i + 1], more) << 16;
    }
    if (code[0] == other[0] && code[1] == other[1]) return;
    float f[8];
    Oct<DT>::unpack(w, f);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        code[i] = e4m3_pair(f2_pack(f[4 * i] / s, f[4 * i + 1] / s), 1.f) |
                  e4m3_pair(f2_pack(f[4 * i + 2] / s, f[4 * i + 3] / s), 1.f) << 16;
}

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 3) quant_weight_blocks(const WeightArgs a) {
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
        const int hi = row0 + kRows * i < a.N ? width : 0;
#pragma unroll
        for (int j = 0; j < W; ++j) v[i][j] = 0u;
        if (hi > 0) octet_load<DT, ALIGNED>(w + i * kRows * a.ldw * EB, 0, hi, v[i]);
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < kOctets; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) m = larger_bits<DT>(m, v[i][j]);
    float amax = warp_allmax(bits_value<DT>(m));
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = warp_allmax(part[lane & (kThreads / 32 - 1)]);
    float s = amax / 448.0f;
    if (s < 1.17549435e-38f) s = 1.17549435e-38f;  // 2^-126; a NaN stays
    if (a.pow2) s = power_of_two_above(s);
    if (threadIdx.x == 0) a.scales[static_cast<int64_t>(blockIdx.x / a.kblocks) * a.ldscales + kb] = s;
    // (infinite scales: 0, for codes of 0 and NaN)
    const float inv = 1.0f / s, less = inv * (1.0f - 0x1p-22f), more = inv * (1.0f + 0x1p-22f);
    const bool first = o == 0, last = o == 15 || col + 8 >= a.K;
    char* out = static_cast<char*>(a.codes) + row0 * a.ldcodes + col;
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
        uint32_t code[2];
        octet_quotients<DT>(v[i], s, less, more, code);
        octet_store<1, 2, ALIGNED>(out + i * kRows * a.ldcodes, code, row0 + kRows * i < a.N ? width : 0, first, last);
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
