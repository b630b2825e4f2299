// quant.cu -- residual addition, RMSNorm and an 8-bit output with scales.
//
// Per row, h, r and y = (h * r) * g as in add.cu (fp32), then per group of
// columns (the whole row, or 32, 64 or 128):
//     scale = max(amax(|y|) / 448, 2^-126)      (448: the largest e4m3)
//     code  = e4m3(y / scale), saturated, to nearest-even
// With pow2 the scale is rounded up to a power of two. The floor keeps 1 / scale
// finite for rows of zeros. A NaN anywhere in a group makes its scale NaN; an
// infinity makes the scale infinite, so the group's codes are 0 or NaN.
//
// Bound by HBM (x, residual in; h out; a byte a code), without a residual by
// instructions: converting, scaling and packing 8 columns takes some 100. Measured on
// GB300 (a device copy moves 6.77 TB/s): 16384 x 8192 bf16 with residual 134.5 us (7.0
// TB/s), 8192 x 5120 fp16 without 29.2 us (4.3 TB/s), 64 x 8192 2.7 us a call in a graph.
// Four octets a thread, 139 us against 148 with two, before the sum and the maximum were
// reduced together.
#include "fused.h"
#include "launch.h"
#include "octet.cuh"
#include "quant.cuh"

namespace rmsnorm {

// A block (G == 0) or a warp (G == 32) per row; KB octets per thread. The lanes of a
// group of 32, 64 or 128 columns are 4, 8 or 16 neighbours. With z = h * g a group's
// largest |y| is r times its largest |z|, so the sum of squares and, for a whole row,
// the maximum are reduced together, with one barrier.
template <int DT, int MODE, int G, int KB>
__global__ void __launch_bounds__(G > 0 ? kFusedGroupThreads : G < 0 ? kFusedWideThreads : kFusedMaxThreads) quant_rows(const AddArgs a) {
    constexpr bool AL = MODE == kRowsAligned;
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    __shared__ float part[32];
    __shared__ float top[32];
    const int per_row = G > 0 ? G : blockDim.x;
    const int t = G > 0 ? threadIdx.x % G : threadIdx.x;
    const int lane = threadIdx.x & 31;
    const int64_t row = G > 0 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / G) + threadIdx.x / G : blockIdx.x;
    griddep_wait();
    const bool live = row < a.M;
    const char* xr = static_cast<const char*>(a.x) + row * a.ldx * EB;
    const char* rr = static_cast<const char*>(a.res) + row * a.ldres * EB;
    const char* gr = static_cast<const char*>(a.gamma);

    char* hr = static_cast<char*>(a.h) + row * a.ldh * EB;
    // octets follow the rows of x, residual and h where these share their offset
    const int phase = MODE == kRowsOnePhase ? word_phase<DT>(xr) : 0;

    uint32_t xw[KB][W], rw[KB][W], gw[KB][W];
    Cut cut[KB];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        cut[v] = AL ? whole_cut(v * per_row + t, live ? a.N : 0) : Cut(v * per_row + t, phase, a.N);
        if (!AL && !live) cut[v].hi = 0;
        if constexpr (!AL) {
#pragma unroll
            for (int i = 0; i < W; ++i) xw[v][i] = 0u;
        }
        if (cut[v].live()) row_load<DT, MODE>(xr + cut[v].col * EB, cut[v].lo, cut[v].hi, xw[v]);
    }
    if (a.res) {
#pragma unroll
        for (int v = 0; v < KB; ++v)
            if (cut[v].live()) row_load<DT, MODE>(rr + cut[v].col * EB, cut[v].lo, cut[v].hi, rw[v]);
    }
#pragma unroll
    for (int v = 0; v < KB; ++v)
        if (cut[v].live()) octet_load<DT, AL>(gr + cut[v].col * EB, cut[v].lo, cut[v].hi, gw[v]);

    const uint64_t one2 = f2_pack(a.one, a.one);
    uint64_t ss = f2_pack(0.f, 0.f);
    uint64_t z[KB][4];
    float m[KB];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        m[v] = 0.f;
        if constexpr (!AL) {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[v][e] = 0ull;
        }
        if (cut[v].live()) {
            uint64_t g[4];
            octet_pairs<DT>(xw[v], z[v]);
            if (a.res) {
                uint64_t b[4];
                octet_pairs<DT>(rw[v], b);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[v][e] = f2_add(z[v][e], b[e]);
                pairs_octet<DT>(z[v], xw[v]);
                octet_pairs<DT>(xw[v], z[v]);
            }
            octet_pairs<DT>(gw[v], g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ss = f2_fma(z[v][e], z[v][e], ss);
                z[v][e] = f2_mul(z[v][e], f2_add(g[e], one2));
            }
            m[v] = octet_amax<AL>(z[v], cut[v].lo, cut[v].hi);
        }
        if (a.h && (!AL || cut[v].live()))
            octet_put<DT, AL>(hr + cut[v].col * EB, xw[v], cut[v].lo, cut[v].hi, MODE == kRowsOnePhase, lane == 0,
                              lane == 31 || cut[v].col + 8 >= a.N);
    }
    if (a.group == 0) {
        float all = m[0];
#pragma unroll
        for (int v = 1; v < KB; ++v) all = max_magnitude(all, m[v]);
        all = warp_allmax(all);
        if (G <= 0 && lane == 0) top[threadIdx.x >> 5] = all;  // read after row_sum's barrier
#pragma unroll
        for (int v = 0; v < KB; ++v) m[v] = all;
    } else {
        for (int o = 1; o < 1 << a.group_shift; o <<= 1) {
#pragma unroll
            for (int v = 0; v < KB; ++v) m[v] = max_magnitude(m[v], __shfl_xor_sync(0xffffffffu, m[v], o));
        }
    }
    float s0, s1;
    f2_unpack(ss, s0, s1);
    const float r = row_rsqrt(row_sum<G>(s0 + s1, part), a.inv_n, a.eps);
    if (G <= 0 && a.group == 0) {
        const float all = warp_allmax(lane < static_cast<int>(blockDim.x >> 5) ? top[lane] : 0.f);
#pragma unroll
        for (int v = 0; v < KB; ++v) m[v] = all;
    }
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        quant_store<AL>(a, row, v * per_row + t, cut[v], z[v], m[v], r, lane == 0,
                        lane == 31 || cut[v].col + 8 >= a.N);
    }
    griddep_launch_dependents();
}

template <int DT, int MODE>
static const void* quant_rows_for(int lanes, int octets) {
#define RMSNORM_QUANT_ROWS(G, KB) \
    if (lanes == G && octets == KB) return reinterpret_cast<const void*>(&quant_rows<DT, MODE, G, KB>);
    RMSNORM_QUANT_ROWS(32, 1)
    RMSNORM_QUANT_ROWS(32, 2)
    if constexpr (MODE != kRowsOnePhase) {  // blocks take such rows from 65 octets on
        RMSNORM_QUANT_ROWS(32, 4)
    }
    RMSNORM_QUANT_ROWS(0, 2)
    if constexpr (MODE == kRowsAligned) {
        RMSNORM_QUANT_ROWS(0, 4)
    } else {
        RMSNORM_QUANT_ROWS(-1, 2)
        RMSNORM_QUANT_ROWS(-1, 3)
    }
#undef RMSNORM_QUANT_ROWS
    return nullptr;
}
template <int DT>
static const void* quant_mode(const AddPlan& p) {
    switch (p.mode) {
    case kRowsAligned: return quant_rows_for<DT, kRowsAligned>(p.lanes, p.octets);
    case kRowsOnePhase: return quant_rows_for<DT, kRowsOnePhase>(p.lanes, p.octets);
    default: return quant_rows_for<DT, kRowsAny>(p.lanes, p.octets);
    }
}

const void* quant_kernel(const AddPlan& p) {
    switch (p.dtype) {
    case kF32: return quant_mode<kF32>(p);
    case kF16: return quant_mode<kF16>(p);
    case kBF16: return quant_mode<kBF16>(p);
    default: return nullptr;
    }
}

}  // namespace rmsnorm
