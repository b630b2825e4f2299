// add.cu -- residual addition with dropout and the RMSNorm of the sum: the forward.
//
// Per row, with D(x) = x * scale where the dropout keeps an element and 0 where it
// drops it (D(x) = x without dropout):
//     h = D(x) + residual, rounded to the I/O dtype: the residual stream
//     r = 1 / sqrt(sum(h^2) / N + eps);   y = (h * r) * g
// The norm is taken of the rounded h, so that y is the RMSNorm of what the caller
// holds and the backward, which reads h, differentiates the forward at the point
// where it was evaluated. Arithmetic is fp32; h and y are rounded once.
//
// The dropout mask is never stored: each direction draws an octet's numbers from
// its row and column (octet.cuh).
//
// Bound by HBM: x and residual in, h and y out, 4 M N elements. A row's loads go out at
// once and nothing is staged: with some 30-60 registers a thread the SM holds enough
// rows to keep the memory busy, and blocks that end balance themselves over the SMs.
// Measured on GB300, where a device copy moves 6.77 TB/s: 16384 x 4096 bf16 77 us (6.95
// TB/s), 78.3 us with dropout (four octets a thread; two: 84.4); the same through a
// TMA ring of persistent blocks, 83.6 us. 8192 x 4099 fp16, every row at another offset:
// 53.9 us (5.0 TB/s, bound by instructions: the weight has to be shifted to each row, and the
// divisions and root of r cost 1.4 us; the ring 71-107 us, several rows a block 60 us). 8 x
// 4096: 1.8 us a call in a graph.
#include "fused.h"
#include "launch.h"
#include "octet.cuh"

namespace rmsnorm {

// G lanes per row (several rows per block), or a block per row (0, wide -1); KB octets
// per thread, thread t of a row owning octets t, t + threads, ... Each block does its
// rows and ends: the hardware balances the rows over the SMs, and a row's loads are
// all in flight at once.
template <int DT, int MODE, int G, int KB, bool DROP>
__global__ void __launch_bounds__(G > 0 ? kFusedGroupThreads : G < 0 ? kFusedWideThreads : kFusedMaxThreads) add_fwd_rows(const AddArgs a) {
    constexpr bool AL = MODE == kRowsAligned;
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    __shared__ float part[32];
    const int per_row = G > 0 ? G : blockDim.x;
    const int t = G > 0 ? threadIdx.x % G : threadIdx.x;
    const int64_t row = G > 0 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / G) + threadIdx.x / G : blockIdx.x;
    griddep_wait();
    const bool live = row < a.M;
    const char* xr = static_cast<const char*>(a.x) + row * a.ldx * EB;
    const char* rr = static_cast<const char*>(a.res) + row * a.ldres * EB;
    char* hr = static_cast<char*>(a.h) + row * a.ldh * EB;
    char* yr = static_cast<char*>(a.y) + row * a.ldy * EB;
    const char* gr = static_cast<const char*>(a.gamma);
    const bool on_word = MODE == kRowsOnePhase || a.same_phase != 0;
    const int phase = !AL && on_word ? word_phase<DT>(yr) : 0;

    uint32_t xw[KB][W], rw[KB][W], gw[KB][W];
    Cut cut[KB];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        cut[v] = Cut(v * per_row + t, phase, a.N);
        if (!live) cut[v].hi = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) xw[v][i] = 0u;
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

    const Dropout drop = {a.rng, a.threshold, a.scale};
    PhiloxKey key = {};
    if (DROP) {
        key = philox_key(drop);
        if (a.rng_used && blockIdx.x == 0 && threadIdx.x == 0) {
            a.rng_used[0] = a.rng[0];
            a.rng_used[1] = a.rng[1];
        }
    }
    uint64_t ss = f2_pack(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        if (cut[v].live()) {
            uint64_t f[4];
            octet_pairs<DT>(xw[v], f);
            if (DROP) dropout_octet<!AL>(drop, key, cut[v].col, static_cast<uint32_t>(row), f);
            if (a.res) {
                uint64_t b[4];
                octet_pairs<DT>(rw[v], b);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = f2_add(f[e], b[e]);
            }
            pairs_octet<DT>(f, xw[v]);  // h from here on
            octet_pairs<DT>(xw[v], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = f2_fma(f[e], f[e], ss);
        }
    }
    if (a.h) {
#pragma unroll
        for (int v = 0; v < KB; ++v)
            octet_put<DT, AL>(hr + cut[v].col * EB, xw[v], cut[v].lo, cut[v].hi, on_word, G > 0 ? t == 0 : t % 32 == 0,
                              t % 32 == 31 || (G > 0 && t == G - 1) || cut[v].col + 8 >= a.N);
    }
    float s0, s1;
    f2_unpack(ss, s0, s1);
    // as the library's other norms have it: y is theirs of h but for the order of the sum
    const float r = 1.0f / sqrtf(row_sum<G>(s0 + s1, part) / static_cast<float>(a.N) + a.eps);
    if (live && t == 0 && a.rstd) a.rstd[row] = r;
    const uint64_t r2 = f2_pack(r, r), one2 = f2_pack(1.f, 1.f);
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        if (cut[v].live()) {
            uint64_t f[4], g[4];
            octet_pairs<DT>(xw[v], f);
            octet_pairs<DT>(gw[v], g);
            if (a.one != 0.f) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = f2_mul(f2_mul(f2_add(g[e], one2), f[e]), r2);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = f2_mul(f2_mul(f[e], r2), g[e]);
            }
            pairs_octet<DT>(f, xw[v]);
        }
        octet_put<DT, AL>(yr + cut[v].col * EB, xw[v], cut[v].lo, cut[v].hi, on_word, G > 0 ? t == 0 : t % 32 == 0,
                          t % 32 == 31 || (G > 0 && t == G - 1) || cut[v].col + 8 >= a.N);
    }
    griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
template <int DT, int MODE, bool DROP>
static const void* add_fwd_for(int lanes, int octets) {
#define RMSNORM_ADD_FWD(G, KB) \
    if (lanes == G && octets == KB) return reinterpret_cast<const void*>(&add_fwd_rows<DT, MODE, G, KB, DROP>);
    RMSNORM_ADD_FWD(8, 1)
    RMSNORM_ADD_FWD(8, 2)
    RMSNORM_ADD_FWD(32, 1)
    RMSNORM_ADD_FWD(32, 2)
    if constexpr (MODE != kRowsOnePhase) {  // blocks take such rows from 65 octets on
        RMSNORM_ADD_FWD(32, 4)
    }
    RMSNORM_ADD_FWD(0, 2)
    if constexpr (MODE == kRowsAligned) {
        RMSNORM_ADD_FWD(0, 4)
    } else {
        RMSNORM_ADD_FWD(-1, 2)
        RMSNORM_ADD_FWD(-1, 3)
    }
#undef RMSNORM_ADD_FWD
    return nullptr;
}
template <int DT, bool DROP>
static const void* add_fwd_mode(const AddPlan& p) {
    switch (p.mode) {
    case kRowsAligned: return add_fwd_for<DT, kRowsAligned, DROP>(p.lanes, p.octets);
    case kRowsOnePhase: return add_fwd_for<DT, kRowsOnePhase, DROP>(p.lanes, p.octets);
    default: return add_fwd_for<DT, kRowsAny, DROP>(p.lanes, p.octets);
    }
}

const void* add_fwd_kernel(const AddPlan& p) {
    switch (p.dtype) {
    case kF32: return p.drop ? add_fwd_mode<kF32, true>(p) : add_fwd_mode<kF32, false>(p);
    case kF16: return p.drop ? add_fwd_mode<kF16, true>(p) : add_fwd_mode<kF16, false>(p);
    case kBF16: return p.drop ? add_fwd_mode<kBF16, true>(p) : add_fwd_mode<kBF16, false>(p);
    default: return nullptr;
    }
}

}  // namespace rmsnorm
