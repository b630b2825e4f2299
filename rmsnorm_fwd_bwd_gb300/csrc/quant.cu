// quant.cu -- residual addition, RMSNorm and an 8-bit output with scales.
//
// Per row, h, r and y = (h * r) * g as in add.cu (y stays fp32), then per group of
// columns (the whole row, or 32, 64 or 128):
//     scale = max(amax(|y|) / 448, 2^-126)      (448: the largest e4m3)
//     code  = e4m3(y * (1 / scale)), saturated, to nearest-even
// With pow2 the scale is rounded up to a power of two. The floor keeps 1 / scale
// finite for rows of zeros. A NaN anywhere in a group makes its scale NaN; an
// infinity makes the scale infinite, so the group's codes are 0 or NaN.
#include "fused.h"
#include "launch.h"
#include "octet.cuh"
#include "quant.cuh"

namespace rmsnorm {

// A block (G == 0) or a warp (G == 32) per row; KB octets per thread. The lanes of a
// group of 32, 64 or 128 columns are 4, 8 or 16 neighbours.
template <int DT, bool AL, int G, int KB>
__global__ void __launch_bounds__(G ? kFusedGroupThreads : kFusedMaxThreads) quant_rows(const AddArgs a) {
    using O = Oct<DT>;
    constexpr int W = O::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    __shared__ float part[32];
    __shared__ uint32_t top[32];
    const int per_row = G ? G : blockDim.x;
    const int t = G ? threadIdx.x % G : threadIdx.x;
    const int lane = threadIdx.x & 31;
    const int64_t row = G ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / G) + threadIdx.x / G : blockIdx.x;
    griddep_wait();
    const bool live = row < a.M;
    const char* xr = static_cast<const char*>(a.x) + row * a.ldx * EB;
    const char* rr = static_cast<const char*>(a.res) + row * a.ldres * EB;
    const char* gr = static_cast<const char*>(a.gamma);

    uint32_t xw[KB][W], rw[KB][W], gw[KB][W];
    int valid[KB];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const int o = v * per_row + t;
        valid[v] = live ? Cut(o, 0, a.N).hi : 0;
#pragma unroll
        for (int i = 0; i < W; ++i) xw[v][i] = 0u;
        if (valid[v] > 0) octet_load<DT, AL>(xr + o * O::kBytes, 0, valid[v], xw[v]);
    }
    if (a.res) {
#pragma unroll
        for (int v = 0; v < KB; ++v)
            if (valid[v] > 0) octet_load<DT, AL>(rr + (v * per_row + t) * O::kBytes, 0, valid[v], rw[v]);
    }
#pragma unroll
    for (int v = 0; v < KB; ++v)
        if (valid[v] > 0) octet_load<DT, AL>(gr + (v * per_row + t) * O::kBytes, 0, valid[v], gw[v]);

    uint64_t ss = f2_pack(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const int o = v * per_row + t;
        if (valid[v] > 0) {
            uint64_t f[4];
            octet_pairs<DT>(xw[v], f);
            if (a.res) {
                uint64_t b[4];
                octet_pairs<DT>(rw[v], b);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = f2_add(f[e], b[e]);
                pairs_octet<DT>(f, xw[v]);
                octet_pairs<DT>(xw[v], f);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = f2_fma(f[e], f[e], ss);
        }
        if (a.h && (!AL || valid[v] > 0))
            octet_store<EB, W, AL>(static_cast<char*>(a.h) + row * a.ldh * EB + o * O::kBytes, xw[v], valid[v] * EB,
                                   lane == 0, lane == 31 || 8 * (o + 1) >= a.N);
    }
    float s0, s1;
    f2_unpack(ss, s0, s1);
    const float r = row_rsqrt(row_sum<G>(s0 + s1, part), a.inv_n, a.eps);
    const uint64_t r2 = f2_pack(r, r), one2 = f2_pack(a.one, a.one);
    uint64_t y[KB][4];
    uint32_t m[KB];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        m[v] = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[v][e] = 0ull;
        if (valid[v] > 0) {
            uint64_t g[4];
            octet_pairs<DT>(xw[v], y[v]);
            octet_pairs<DT>(gw[v], g);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[v][e] = f2_mul(f2_mul(y[v][e], r2), f2_add(g[e], one2));
            m[v] = octet_amax(y[v], AL ? 8 : valid[v]);
        }
    }
    if (a.group == 0) {
        uint32_t all = m[0];
#pragma unroll
        for (int v = 1; v < KB; ++v) all = max(all, m[v]);
        all = warp_allmax(all);
        if constexpr (G == 0) {
            if (lane == 0) top[threadIdx.x >> 5] = all;
            __syncthreads();
            all = warp_allmax(lane < static_cast<int>(blockDim.x >> 5) ? top[lane] : 0u);
        }
#pragma unroll
        for (int v = 0; v < KB; ++v) m[v] = all;
    } else {
        for (int o = 1; o < a.group / 8; o <<= 1) {
#pragma unroll
            for (int v = 0; v < KB; ++v) m[v] = max(m[v], __shfl_xor_sync(0xffffffffu, m[v], o));
        }
    }
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const int o = v * per_row + t;
        quant_store<AL>(a, row, o, valid[v], y[v], m[v], lane == 0, lane == 31 || 8 * (o + 1) >= a.N);
    }
    griddep_launch_dependents();
}

template <int DT, bool AL>
static const void* quant_rows_for(int lanes, int octets) {
#define RMSNORM_QUANT_ROWS(G, KB) \
    if (lanes == G && octets == KB) return reinterpret_cast<const void*>(&quant_rows<DT, AL, G, KB>);
    RMSNORM_QUANT_ROWS(32, 1)
    RMSNORM_QUANT_ROWS(32, 2)
    RMSNORM_QUANT_ROWS(32, 4)
    RMSNORM_QUANT_ROWS(0, 1)
    RMSNORM_QUANT_ROWS(0, 2)
    RMSNORM_QUANT_ROWS(0, 4)
#undef RMSNORM_QUANT_ROWS
    return nullptr;
}

const void* quant_kernel(const AddPlan& p) {
    switch (p.dtype) {
    case kF32: return p.aligned ? quant_rows_for<kF32, true>(p.lanes, p.octets) : quant_rows_for<kF32, false>(p.lanes, p.octets);
    case kF16: return p.aligned ? quant_rows_for<kF16, true>(p.lanes, p.octets) : quant_rows_for<kF16, false>(p.lanes, p.octets);
    case kBF16: return p.aligned ? quant_rows_for<kBF16, true>(p.lanes, p.octets) : quant_rows_for<kBF16, false>(p.lanes, p.octets);
    default: return nullptr;
    }
}

}  // namespace rmsnorm
