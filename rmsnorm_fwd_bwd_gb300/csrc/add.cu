// add.cu -- residual addition with dropout and the RMSNorm of the sum, forward and
// backward.
//
// Per row, with D(x) = x * scale where the dropout keeps an element and 0 where it
// drops it (D(x) = x without dropout):
//     h = D(x) + residual, rounded to the I/O dtype: the residual stream
//     r = 1 / sqrt(sum(h^2) / N + eps);   y = (h * r) * g
// and for the cotangents dy of y and dh of h, n = h * r, u = dy * g:
//     dresidual = dh + r * (u - n * (sum(u * n) / N))
//     dx = D'(dresidual)  (the same elements kept, the same scale, before rounding)
//     dgamma = sum over rows of dy * n
// The norm is taken of the rounded h, so that y is the RMSNorm of what the caller
// holds and the backward, which reads h, differentiates the forward at the point
// where it was evaluated. Arithmetic is fp32; h, y, dresidual and dx are rounded
// once.
//
// The dropout mask is never stored: each direction draws an octet's numbers from
// its row and column (octet.cuh).
#include "fused.h"
#include "launch.h"
#include "octet.cuh"

namespace rmsnorm {

// Forward. G lanes per row (several rows per block), or a block per row (G == 0);
// KB octets per thread, thread t of a row owning octets t, t + threads, ... Each
// block does its rows and ends: the hardware balances the rows over the SMs.
template <int DT, bool AL, int G, int KB>
__global__ void __launch_bounds__(G ? kFusedGroupThreads : kFusedMaxThreads) add_fwd_rows(const AddArgs a) {
    using O = Oct<DT>;
    constexpr int W = O::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    __shared__ float part[32];
    const int per_row = G ? G : blockDim.x;
    const int t = G ? threadIdx.x % G : threadIdx.x;
    const int64_t row = G ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / G) + threadIdx.x / G : blockIdx.x;
    const bool first = G ? t == 0 : (t & 31) == 0;
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

    const Dropout drop = {a.rng, a.threshold, a.scale};
    PhiloxKey key = {};
    if (a.threshold) {
        key = philox_key(drop);
        if (a.rng_used && blockIdx.x == 0 && threadIdx.x == 0) {
            a.rng_used[0] = a.rng[0];
            a.rng_used[1] = a.rng[1];
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const int o = v * per_row + t;
        if (valid[v] > 0) {
            float f[8];
            O::unpack(xw[v], f);
            if (a.threshold) dropout_octet(drop, key, o, static_cast<uint32_t>(row), f);
            if (a.res) {
                float b[8];
                O::unpack(rw[v], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] += b[e];
            }
            O::pack(f, xw[v]);  // h from here on
            O::unpack(xw[v], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
        }
        if (a.h && (!AL || valid[v] > 0))
            octet_store<EB, W, AL>(static_cast<char*>(a.h) + row * a.ldh * EB + o * O::kBytes, xw[v], valid[v] * EB,
                                   first, t % 32 == 31 || (G && t == G - 1) || 8 * (o + 1) >= a.N);
    }
    ss = row_sum<G>(ss, part);
    const float r = 1.0f / sqrtf(ss / static_cast<float>(a.N) + a.eps);
    if (live && t == 0 && a.rstd) a.rstd[row] = r;
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const int o = v * per_row + t;
        if (valid[v] > 0) {
            float f[8], g[8];
            O::unpack(xw[v], f);
            O::unpack(gw[v], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (f[e] * r) * (g[e] + a.one);
            O::pack(f, xw[v]);
        }
        if (!AL || valid[v] > 0)
            octet_store<EB, W, AL>(static_cast<char*>(a.y) + row * a.ldy * EB + o * O::kBytes, xw[v], valid[v] * EB,
                                   first, t % 32 == 31 || (G && t == G - 1) || 8 * (o + 1) >= a.N);
    }
    griddep_launch_dependents();
}

// Backward: persistent, so that a thread, which owns the same columns in all its
// rows, adds their share of dgamma up in registers. A block's rows (G == 0) or its
// groups' rows are a fixed set in a fixed order, and each block writes one row of
// partial sums for the fixed-order column reduce: dgamma is deterministic.
template <int DT, bool AL, int G, int KB>
__global__ void __launch_bounds__(G ? kFusedGroupThreads : kFusedMaxThreads) add_bwd_rows(const AddArgs a) {
    using O = Oct<DT>;
    constexpr int W = O::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    __shared__ float part[2][32];
    extern __shared__ float sums[];  // G > 0: [groups of the block][N]
    const int per_row = G ? G : blockDim.x;
    const int rows_block = G ? blockDim.x / G : 1;
    const int t = G ? threadIdx.x % G : threadIdx.x;
    const bool first = G ? t == 0 : (t & 31) == 0;
    const char* gr = static_cast<const char*>(a.gamma);
    griddep_wait();

    uint32_t gw[KB][W];
    float acc[KB][8];
    int valid[KB];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const int o = v * per_row + t;
        valid[v] = octet_valid(o, a.N);
        if (valid[v] > 0) octet_load<DT, AL>(gr + o * O::kBytes, valid[v], gw[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[v][e] = 0.f;
    }
    const Dropout drop = {a.rng, a.threshold, a.scale};
    PhiloxKey key = {};
    if (a.threshold) key = philox_key(drop);
    const float inv_n = 1.0f / static_cast<float>(a.N);

    int parity = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_block;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows_block; base < a.M; base += step, parity ^= 1) {
        const int64_t row = base + (G ? threadIdx.x / G : 0);
        const bool live = row < a.M;
        const char* dyr = static_cast<const char*>(a.dy) + row * a.lddy * EB;
        const char* hr = static_cast<const char*>(a.x) + row * a.ldx * EB;
        const char* dhr = static_cast<const char*>(a.dh) + row * a.lddh * EB;
        const float r = live ? a.rstd[row] : 0.f;
        uint32_t yw[KB][W], hw[KB][W], ew[KB][W];
#pragma unroll
        for (int v = 0; v < KB; ++v) {
            const int o = v * per_row + t;
            const int n = live ? valid[v] : 0;
#pragma unroll
            for (int i = 0; i < W; ++i) yw[v][i] = hw[v][i] = ew[v][i] = 0u;
            if (n > 0) {
                octet_load<DT, AL>(dyr + o * O::kBytes, n, yw[v]);
                octet_load<DT, AL>(hr + o * O::kBytes, n, hw[v]);
                if (a.dh) octet_load<DT, AL>(dhr + o * O::kBytes, n, ew[v]);
            }
        }
        float c = 0.f;
#pragma unroll
        for (int v = 0; v < KB; ++v) {
            if (valid[v] > 0) {
                float d[8], h[8], g[8];
                O::unpack(yw[v], d);
                O::unpack(hw[v], h);
                O::unpack(gw[v], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = h[e] * r;
                    const float w = d[e] * n;
                    acc[v][e] += w;
                    c = fmaf(w, g[e] + a.one, c);
                }
            }
        }
        c = row_sum<G>(c, part[parity]) * inv_n;
#pragma unroll
        for (int v = 0; v < KB; ++v) {
            const int o = v * per_row + t;
            const int n = live ? valid[v] : 0;
            const bool last = t % 32 == 31 || (G && t == G - 1) || 8 * (o + 1) >= a.N;
            float d[8], h[8], g[8];
            if (n > 0) {
                float q[8];
                O::unpack(yw[v], d);
                O::unpack(hw[v], h);
                O::unpack(gw[v], g);
                O::unpack(ew[v], q);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    d[e] = fmaf(r, fmaf(-(h[e] * r), c, d[e] * (g[e] + a.one)), q[e]);
                O::pack(d, yw[v]);
            }
            if (a.dres && (!AL || n > 0))
                octet_store<EB, W, AL>(static_cast<char*>(a.dres) + row * a.lddres * EB + o * O::kBytes, yw[v], n * EB,
                                       first, last);
            if (a.dx) {
                if (n > 0 && a.threshold) {
                    dropout_octet(drop, key, o, static_cast<uint32_t>(row), d);
                    O::pack(d, yw[v]);
                }
                if (!AL || n > 0)
                    octet_store<EB, W, AL>(static_cast<char*>(a.dx) + row * a.lddx * EB + o * O::kBytes, yw[v], n * EB,
                                           first, last);
            }
        }
    }
    // this block's partial row
    float* out = a.ws + static_cast<int64_t>(blockIdx.x) * a.ldws;
    if constexpr (G > 0) {
#pragma unroll
        for (int v = 0; v < KB; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < valid[v]) sums[(threadIdx.x / G) * a.N + 8 * (v * per_row + t) + e] = acc[v][e];
        __syncthreads();
        for (int col = threadIdx.x; col < a.N; col += blockDim.x) {
            float s = sums[col];
            for (int k = 1; k < rows_block; ++k) s += sums[k * a.N + col];
            out[col] = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < KB; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < valid[v]) out[8 * (v * per_row + t) + e] = acc[v][e];
    }
    griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
template <int DT, bool AL, bool BWD>
static const void* add_rows_for(int lanes, int octets) {
#define RMSNORM_ADD_ROWS(G, KB)                                                          \
    if (lanes == G && octets == KB)                                                      \
        return BWD ? reinterpret_cast<const void*>(&add_bwd_rows<DT, AL, G, KB>)         \
                   : reinterpret_cast<const void*>(&add_fwd_rows<DT, AL, G, KB>);
    RMSNORM_ADD_ROWS(8, 1)
    RMSNORM_ADD_ROWS(8, 2)
    RMSNORM_ADD_ROWS(32, 1)
    RMSNORM_ADD_ROWS(32, 2)
    RMSNORM_ADD_ROWS(32, 4)
    RMSNORM_ADD_ROWS(0, 1)
    RMSNORM_ADD_ROWS(0, 2)
    RMSNORM_ADD_ROWS(0, 4)
#undef RMSNORM_ADD_ROWS
    return nullptr;
}
template <bool BWD>
static const void* add_rows(const AddPlan& p) {
    switch (p.dtype) {
    case kF32: return p.aligned ? add_rows_for<kF32, true, BWD>(p.lanes, p.octets) : add_rows_for<kF32, false, BWD>(p.lanes, p.octets);
    case kF16: return p.aligned ? add_rows_for<kF16, true, BWD>(p.lanes, p.octets) : add_rows_for<kF16, false, BWD>(p.lanes, p.octets);
    case kBF16: return p.aligned ? add_rows_for<kBF16, true, BWD>(p.lanes, p.octets) : add_rows_for<kBF16, false, BWD>(p.lanes, p.octets);
    default: return nullptr;
    }
}

const void* add_fwd_kernel(const AddPlan& p) { return add_rows<false>(p); }
const void* add_bwd_kernel(const AddPlan& p) { return add_rows<true>(p); }

}  // namespace rmsnorm
