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

namespace rmsnorm {

// Two fp32 values as e4m3, a in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(b), "f"(a));
    return v;
}

// |y| as an integer: ordered as the value, with NaN above infinity.
__device__ __forceinline__ uint32_t magnitude(float y) { return __float_as_uint(y) & 0x7fffffffu; }

__device__ __forceinline__ float quant_scale(uint32_t amax, int pow2) {
    float s = __uint_as_float(amax) / 448.0f;
    if (s < 1.17549435e-38f) s = 1.17549435e-38f;  // 2^-126; a NaN stays
    if (pow2) {
        // up to the next power of two: a carry out of the fraction raises the exponent
        // (infinity and NaN stay)
        const uint32_t b = __float_as_uint(s);
        if (b < 0x7f800000u) s = __uint_as_float((b + 0x007fffffu) & 0x7f800000u);
    }
    return s;
}

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
        valid[v] = live ? octet_valid(o, a.N) : 0;
#pragma unroll
        for (int i = 0; i < W; ++i) xw[v][i] = 0u;
        if (valid[v] > 0) octet_load<DT, AL>(xr + o * O::kBytes, valid[v], xw[v]);
    }
    if (a.res) {
#pragma unroll
        for (int v = 0; v < KB; ++v)
            if (valid[v] > 0) octet_load<DT, AL>(rr + (v * per_row + t) * O::kBytes, valid[v], rw[v]);
    }
#pragma unroll
    for (int v = 0; v < KB; ++v)
        if (valid[v] > 0) octet_load<DT, AL>(gr + (v * per_row + t) * O::kBytes, valid[v], gw[v]);

    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const int o = v * per_row + t;
        if (valid[v] > 0) {
            float f[8];
            O::unpack(xw[v], f);
            if (a.res) {
                float b[8];
                O::unpack(rw[v], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] += b[e];
                O::pack(f, xw[v]);
                O::unpack(xw[v], f);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
        }
        if (a.h && (!AL || valid[v] > 0))
            octet_store<EB, W, AL>(static_cast<char*>(a.h) + row * a.ldh * EB + o * O::kBytes, xw[v], valid[v] * EB,
                                   lane == 0, lane == 31 || 8 * (o + 1) >= a.N);
    }
    ss = row_sum<G>(ss, part);
    const float r = 1.0f / sqrtf(ss / static_cast<float>(a.N) + a.eps);
    float y[KB][8];
    uint32_t m[KB];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        m[v] = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[v][e] = 0.f;
        if (valid[v] > 0) {
            float g[8];
            O::unpack(xw[v], y[v]);
            O::unpack(gw[v], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[v][e] = (y[v][e] * r) * (g[e] + a.one);
                if (AL || e < valid[v]) m[v] = max(m[v], magnitude(y[v][e]));
            }
        }
    }
    if (a.group == 0) {
        uint32_t all = m[0];
#pragma unroll
        for (int v = 1; v < KB; ++v) all = max(all, m[v]);
        all = __reduce_max_sync(0xffffffffu, all);
        if constexpr (G == 0) {
            if (lane == 0) top[threadIdx.x >> 5] = all;
            __syncthreads();
            all = __reduce_max_sync(0xffffffffu, lane < static_cast<int>(blockDim.x >> 5) ? top[lane] : 0u);
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
        const float s = quant_scale(m[v], a.pow2);
        const float inv = 1.0f / s;
        uint32_t code[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            code[i] = e4m3_pair(y[v][4 * i] * inv, y[v][4 * i + 1] * inv) |
                      e4m3_pair(y[v][4 * i + 2] * inv, y[v][4 * i + 3] * inv) << 16;
        if (!AL || valid[v] > 0)
            octet_store<1, 2, AL>(static_cast<char*>(a.y) + row * a.ldy + o * 8, code, valid[v], lane == 0,
                                  lane == 31 || 8 * (o + 1) >= a.N);
        if (valid[v] > 0) {
            float* sr = a.scales + row * a.ldscales;
            if (a.group == 0) {
                if (o == 0) sr[0] = s;
            } else if (o % (a.group / 8) == 0) {
                sr[o / (a.group / 8)] = s;
            }
        }
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
