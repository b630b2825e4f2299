// add_bwd.cu -- backward of the residual addition, its dropout and the RMSNorm.
//
// Per row, for the cotangents dy of y and dh of h, with the forward's h and r,
// n = h * r, u = dy * g and D' the forward's dropout (the same elements, the same
// scale):
//     dresidual = dh + r * (u - n * (sum(u * n) / N))
//     dx = D'(dresidual), before dresidual is rounded
//     dgamma = sum over rows of dy * n
// Arithmetic is fp32; dresidual and dx are rounded once.
//
// Both kernels are persistent, so that a thread, which owns the same columns in all
// its rows, adds their share of dgamma up in registers; a block's rows are a fixed
// set in a fixed order, and each block writes one row of partial sums for the
// fixed-order column reduce: dgamma is deterministic.
//
// Rows off 16 bytes: the grid is a multiple of 8, and rows 8 apart start at the same
// offset from a 16-byte boundary (a pitch is a whole number of 2-byte elements at
// least), so all rows of a thread share theirs and its columns stay the same.
//
// Bound by HBM: dy, dh and h in, dresidual (and dx) out, 4 or 5 M N elements. Measured on
// GB300 (a device copy moves 6.77 TB/s), the column reduction of 5 us in each figure:
// 65536 x 4096 bf16 with dropout 422 us (6.35 TB/s), 16384 x 4096 without 91 us (5.9 TB/s),
// 8192 x 4099 58 us (4.6 TB/s), 65536 x 1000 by lanes 89 us (5.9 TB/s). Without the ring
// the first took 536 us: loads waited for at every row.
#include "fused.h"
#include "launch.h"
#include "octet.cuh"

namespace rmsnorm {

// G lanes per row, or a block per row (G == 0), loads straight into registers: rows
// of up to 1024 elements, wider ones where they are few, and those too wide for the
// ring or not of one offset.
template <int DT, int MODE, int G, int KB>
__global__ void __launch_bounds__(G ? kFusedGroupThreads : kFusedMaxThreads) add_bwd_rows(const AddArgs a) {
    constexpr bool AL = MODE == kRowsAligned;
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    __shared__ float part[2][32];
    extern __shared__ float sums[];  // G > 0: [groups of the block][N]
    const int per_row = G ? G : blockDim.x;
    const int rows_block = G ? blockDim.x / G : 1;
    const int t = G ? threadIdx.x % G : threadIdx.x;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_block + (G ? threadIdx.x / G : 0);
    const bool first = G ? t == 0 : (t & 31) == 0;
    const char* gr = static_cast<const char*>(a.gamma);
    griddep_wait();
    const bool on_word = MODE == kRowsOnePhase || a.same_phase != 0;
    // the offset that octets follow: the one of all tensors, or that of the outputs (of
    // which there may be none)
    const char* follow = static_cast<const char*>(MODE == kRowsOnePhase ? a.dy : a.dres ? a.dres : a.dx);
    const int64_t pitch = MODE == kRowsOnePhase ? a.lddy : a.dres ? a.lddres : a.lddx;
    const int phase = AL || !on_word || !follow ? 0 : word_phase<DT>(follow + row0 * pitch * EB);

    uint32_t gw[KB][W];
    uint64_t acc[KB][4];
    Cut cut[KB];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        cut[v] = Cut(v * per_row + t, phase, a.N);
        if (cut[v].live()) octet_load<DT, AL>(gr + cut[v].col * EB, cut[v].lo, cut[v].hi, gw[v]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[v][e] = f2_pack(0.f, 0.f);
    }
    const Dropout drop = {a.rng, a.threshold, a.scale};
    PhiloxKey key = {};
    if (a.threshold) key = philox_key(drop);
    const float inv_n = 1.0f / static_cast<float>(a.N);
    const uint64_t one2 = f2_pack(a.one, a.one);

    int parity = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_block;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows_block; base < a.M; base += step, parity ^= 1) {
        const int64_t row = base + (G ? threadIdx.x / G : 0);
        const bool live = row < a.M;
        const char* dyr = static_cast<const char*>(a.dy) + row * a.lddy * EB;
        const char* hr = static_cast<const char*>(a.x) + row * a.ldx * EB;
        const char* dhr = static_cast<const char*>(a.dh) + row * a.lddh * EB;
        const float r = live ? a.rstd[row] : 0.f;
        const uint64_t r2 = f2_pack(r, r);
        uint32_t yw[KB][W], hw[KB][W], ew[KB][W];
#pragma unroll
        for (int v = 0; v < KB; ++v) {
#pragma unroll
            for (int i = 0; i < W; ++i) yw[v][i] = hw[v][i] = ew[v][i] = 0u;
            if (live && cut[v].live()) {
                row_load<DT, MODE>(dyr + cut[v].col * EB, cut[v].lo, cut[v].hi, yw[v]);
                row_load<DT, MODE>(hr + cut[v].col * EB, cut[v].lo, cut[v].hi, hw[v]);
                if (a.dh) row_load<DT, MODE>(dhr + cut[v].col * EB, cut[v].lo, cut[v].hi, ew[v]);
            }
        }
        uint64_t c2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < KB; ++v) {
            if (cut[v].live()) {
                uint64_t d[4], h[4], g[4];
                octet_pairs<DT>(yw[v], d);
                octet_pairs<DT>(hw[v], h);
                octet_pairs<DT>(gw[v], g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t w = f2_mul(d[e], f2_mul(h[e], r2));
                    acc[v][e] = f2_add(acc[v][e], w);
                    c2 = f2_fma(w, f2_add(g[e], one2), c2);
                }
            }
        }
        float ca, cb;
        f2_unpack(c2, ca, cb);
        const float m = -(row_sum<G>(ca + cb, part[parity]) * inv_n);  // -mean(u * n)
        const uint64_t m2 = f2_pack(m, m);
#pragma unroll
        for (int v = 0; v < KB; ++v) {
            const bool has = live && cut[v].live();
            const int hi = live ? cut[v].hi : 0;
            const bool last = t % 32 == 31 || (G && t == G - 1) || cut[v].col + 8 >= a.N;
            uint64_t d[4];
            if (has) {
                uint64_t h[4], g[4], q[4];
                octet_pairs<DT>(yw[v], d);
                octet_pairs<DT>(hw[v], h);
                octet_pairs<DT>(gw[v], g);
                octet_pairs<DT>(ew[v], q);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    d[e] = f2_fma(f2_fma(f2_mul(h[e], r2), m2, f2_mul(d[e], f2_add(g[e], one2))), r2, q[e]);
                pairs_octet<DT>(d, yw[v]);
            }
            if (a.dres)
                octet_put<DT, AL>(static_cast<char*>(a.dres) + (row * a.lddres + cut[v].col) * EB, yw[v], cut[v].lo, hi,
                                  on_word, first, last);
            if (a.dx) {
                if (has && a.threshold) {
                    dropout_octet<!AL>(drop, key, cut[v].col, static_cast<uint32_t>(row), d);
                    pairs_octet<DT>(d, yw[v]);
                }
                octet_put<DT, AL>(static_cast<char*>(a.dx) + (row * a.lddx + cut[v].col) * EB, yw[v], cut[v].lo, hi, on_word,
                                  first, last);
            }
        }
    }
    // this block's partial row
    float* out = a.ws + static_cast<int64_t>(blockIdx.x) * a.ldws;
    float* mine = G ? sums + (threadIdx.x / G) * a.N : out;
#pragma unroll
    for (int v = 0; v < KB; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x, y;
            f2_unpack(acc[v][e], x, y);
            if (2 * e >= cut[v].lo && 2 * e < cut[v].hi) mine[cut[v].col + 2 * e] = x;
            if (2 * e + 1 >= cut[v].lo && 2 * e + 1 < cut[v].hi) mine[cut[v].col + 2 * e + 1] = y;
        }
    if constexpr (G > 0) {
        __syncthreads();
        for (int col = threadIdx.x; col < a.N; col += blockDim.x) {
            float s = sums[col];
            for (int k = 1; k < rows_block; ++k) s += sums[k * a.N + col];
            out[col] = s;
        }
    }
    griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// The ring: a block per row, its tensors brought into shared memory by TMA bulk
// copies a few rows ahead. One thread issues a row's copies (dy, h and dh), counted
// by the stage's mbarrier. The kernel is bound by HBM: what it needs is bytes in
// flight all the time, which the ring gives without holding them in registers.
//
// A stage is read twice (the row sum, then the gradients) and refilled one row later,
// when the next row's one block barrier shows that every thread is done with it. Reading
// twice keeps dy and h out of the registers, and packed pairs halve the instructions:
// three blocks of 256 threads fit an SM, where 120 registers left two (bf16 65536 x 4096
// with dropout: 489 -> 423 us).
//
// AL: rows of whole octets on 16-byte boundaries. Otherwise the rows of all tensors
// start at one offset from a 16-byte boundary (the usual dense tensors of any width):
// a copy takes the 16-byte words around a row, octets start on 16-byte boundaries, and
// only a row's two ends are masked.
// ---------------------------------------------------------------------------
namespace {

// An octet in shared memory as four pairs of fp32 values; elements outside [lo, hi) zero.
template <int DT, bool AL>
__device__ __forceinline__ void ring_load(const unsigned char* p, const Cut& c, uint64_t (&f)[4]) {
    constexpr int W = Oct<DT>::kWords;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
    if (!AL && (c.lo > 0 || c.hi < 8)) octet_keep<DT>(w, c.lo, c.hi);
    octet_pairs<DT>(w, f);
}

// The gains of a thread's octets, g or 1 + g, in shared memory: in fp32 where there is
// room (two octets per thread), as four-element halves so that neighbouring lanes read
// neighbouring words; else as they are.
template <int DT, int KB> struct Gains {
    static constexpr bool kWide = KB == 2;
    static constexpr int kBytes = kWide ? 32 : Oct<DT>::kBytes;  // per octet
    unsigned char* at;
    int nt, tid;
    __device__ __forceinline__ void put(int v, const uint32_t (&w)[Oct<DT>::kWords], uint64_t one2) const {
        if constexpr (kWide) {
            uint64_t g[4];
            octet_pairs<DT>(w, g);
            ulonglong2* p = reinterpret_cast<ulonglong2*>(at);
            p[(2 * v) * nt + tid] = make_ulonglong2(f2_add(g[0], one2), f2_add(g[1], one2));
            p[(2 * v + 1) * nt + tid] = make_ulonglong2(f2_add(g[2], one2), f2_add(g[3], one2));
        } else {
#pragma unroll
            for (int i = 0; i < Oct<DT>::kWords / 4; ++i)
                reinterpret_cast<uint4*>(at + (v * nt + tid) * kBytes)[i] =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
    __device__ __forceinline__ void get(int v, uint64_t one2, uint64_t (&g)[4]) const {
        if constexpr (kWide) {
            const ulonglong2* p = reinterpret_cast<const ulonglong2*>(at);
            const ulonglong2 a = p[(2 * v) * nt + tid], b = p[(2 * v + 1) * nt + tid];
            g[0] = a.x; g[1] = a.y; g[2] = b.x; g[3] = b.y;
        } else {
            ring_load<DT, true>(at + (v * nt + tid) * kBytes, Cut(), g);
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = f2_add(g[e], one2);
        }
    }
};

// Registers of a thread: 80 where two octets fit them (three blocks of 256 threads an
// SM), else what 512 threads leave.
template <int KB> struct RingRegisters { static constexpr int value = KB == 2 ? 80 : 128; };

}  // namespace

template <int DT, bool AL, int KB, bool DROP>
__global__ void __maxnreg__((RingRegisters<KB>::value)) add_bwd_ring(const AddArgs a) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x;
    const int nt = blockDim.x;
    const int lane = tid & 31;
    const int warp = tid >> 5;
    const int nwarps = nt >> 5;
    const int S = a.stages;
    const uint32_t stage_bytes = (a.dh ? 3u : 2u) * a.slot;
    // shared memory: ring | gamma's octets, [KB][threads] | full barriers | warp partials [2][32]
    unsigned char* ring = smem;
    unsigned char* gsm = smem + static_cast<size_t>(S) * stage_bytes;
    const Gains<DT, KB> gains = {gsm, nt, tid};
    uint64_t* full = reinterpret_cast<uint64_t*>(gsm + static_cast<size_t>(KB) * nt * Gains<DT, KB>::kBytes);
    float* part = reinterpret_cast<float*>(full + S);
    const int64_t G = gridDim.x;
    const int64_t nrows = blockIdx.x < a.M ? (a.M - 1 - blockIdx.x) / G + 1 : 0;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init(smem_u32(&full[s]), 1);
        fence_mbar_init();
    }
    griddep_wait();  // inputs may come from the previous kernel on the stream
    const uint64_t pol = l2_evict_first_policy();
    // the rows' offset from a 16-byte boundary, and a row's copy
    const uint32_t shift = AL ? 0u : static_cast<uint32_t>((reinterpret_cast<uintptr_t>(a.dy) + blockIdx.x * a.lddy * EB) & 15);
    const uint32_t bytes = AL ? static_cast<uint32_t>(a.N * EB) : (shift + static_cast<uint32_t>(a.N * EB) + 15u) & ~15u;
    auto fill = [&](int64_t j) {
        const int s = static_cast<int>(j % S);
        const int64_t row = blockIdx.x + j * G;
        const uint32_t bar = smem_u32(&full[s]);
        const uint32_t slot = smem_u32(ring + static_cast<size_t>(s) * stage_bytes);
        mbar_arrive_expect_tx(bar, a.dh ? 3 * bytes : 2 * bytes);
        bulk_g2s_in(slot, static_cast<const char*>(a.dy) + row * a.lddy * EB - shift, bytes, bar, pol, a.dy, a.M, a.lddy, a.N,
                    EB, a.err);
        bulk_g2s_in(slot + a.slot, static_cast<const char*>(a.x) + row * a.ldx * EB - shift, bytes, bar, pol, a.x, a.M,
                    a.ldx, a.N, EB, a.err);
        if (a.dh)
            bulk_g2s_in(slot + 2 * a.slot, static_cast<const char*>(a.dh) + row * a.lddh * EB - shift, bytes, bar, pol, a.dh,
                        a.M, a.lddh, a.N, EB, a.err);
    };
    if (tid == 0)
        for (int64_t j = 0; j < (nrows < S ? nrows : S); ++j) fill(j);

    const int phase = static_cast<int>(shift) / EB;
    auto cut_of = [&](int v) {
        Cut c(v * nt + tid, phase, a.N);
        if (AL) {
            c.lo = 0;
            c.hi = c.col < a.N ? 8 : 0;
        }
        return c;
    };
    const uint64_t one2 = f2_pack(a.one, a.one);
    uint64_t acc[KB][4];
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const Cut c = cut_of(v);
        uint32_t g[W];
#pragma unroll
        for (int i = 0; i < W; ++i) g[i] = 0u;
        if (c.live()) octet_load<DT, AL>(static_cast<const char*>(a.gamma) + c.col * EB, c.lo, c.hi, g);
        gains.put(v, g, one2);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[v][e] = f2_pack(0.f, 0.f);
    }
    const Dropout drop = {a.rng, a.threshold, a.scale};
    PhiloxKey key = {};
    if (DROP) key = philox_key(drop);
    const float inv_n = 1.0f / static_cast<float>(a.N);
    float r_next = nrows > 0 ? a.rstd[blockIdx.x] : 0.f;
    __syncthreads();

    int64_t j = 0;
    int s = 0;
    uint32_t parity = 0;
    bool aborted = false;
    for (; j < nrows; ++j) {
        const int64_t row = blockIdx.x + j * G;
        const unsigned char* slot = ring + static_cast<size_t>(s) * stage_bytes;
        const float r = r_next;
        const uint64_t r2 = f2_pack(r, r);
        if (j + 1 < nrows) r_next = a.rstd[row + G];
        const bool landed = mbar_wait_bounded(smem_u32(&full[s]), parity, a.err);
        uint64_t c2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < KB; ++v) {
            const Cut c = cut_of(v);
            if (c.live()) {
                const unsigned char* p = slot + (v * nt + tid) * Oct<DT>::kBytes;
                uint64_t d[4], h[4], g[4];
                ring_load<DT, AL>(p, c, d);
                ring_load<DT, AL>(p + a.slot, c, h);
                gains.get(v, one2, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t w = f2_mul(d[e], f2_mul(h[e], r2));
                    acc[v][e] = f2_add(acc[v][e], w);
                    c2 = f2_fma(w, g[e], c2);
                }
            }
        }
        float ca, cb;
        f2_unpack(c2, ca, cb);
        float* partj = part + (j & 1) * 32;
        ca = warp_allsum(ca + cb);
        if (lane == 0) partj[warp] = ca;
        // the row's partial sums; and every thread is done with the row before
        if (__syncthreads_or(!landed)) {
            aborted = true;
            break;
        }
        if (tid == 0 && j > 0 && j - 1 + S < nrows) {
            fence_proxy_async_smem();
            fill(j - 1 + S);
        }
        // -mean(u * n): the gradient is dh + r * (u - n * mean)
        const float m = -(warp_allsum(lane < nwarps ? partj[lane] : 0.f) * inv_n);
        const uint64_t m2 = f2_pack(m, m);
#pragma unroll
        for (int v = 0; v < KB; ++v) {
            const Cut c = cut_of(v);
            if (c.live()) {
                const unsigned char* p = slot + (v * nt + tid) * Oct<DT>::kBytes;
                uint64_t d[4], h[4], g[4];
                ring_load<DT, true>(p, c, d);
                ring_load<DT, true>(p + a.slot, c, h);
                gains.get(v, one2, g);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    d[e] = f2_fma(f2_mul(h[e], r2), m2, f2_mul(d[e], g[e]));
                if (a.dh) {
                    ring_load<DT, true>(p + 2 * a.slot, c, g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = f2_fma(d[e], r2, g[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = f2_mul(d[e], r2);
                }
                uint32_t w[W];
                if (a.dres) {
                    pairs_octet<DT>(d, w);
                    octet_put<DT, AL>(static_cast<char*>(a.dres) + (row * a.lddres + c.col) * EB, w, c.lo, c.hi, true, false,
                                      false);
                }
                if (a.dx) {
                    if (DROP) dropout_octet<!AL>(drop, key, c.col, static_cast<uint32_t>(row), d);
                    pairs_octet<DT>(d, w);
                    octet_put<DT, AL>(static_cast<char*>(a.dx) + (row * a.lddx + c.col) * EB, w, c.lo, c.hi, true, false,
                                      false);
                }
            }
        }
        if (++s == S) {
            s = 0;
            parity ^= 1u;
        }
    }
    // this block's partial row
    float* out = a.ws + static_cast<int64_t>(blockIdx.x) * a.ldws;
#pragma unroll
    for (int v = 0; v < KB; ++v) {
        const Cut c = cut_of(v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x, y;
            f2_unpack(acc[v][e], x, y);
            if (2 * e >= c.lo && 2 * e < c.hi) out[c.col + 2 * e] = x;
            if (2 * e + 1 >= c.lo && 2 * e + 1 < c.hi) out[c.col + 2 * e + 1] = y;
        }
    }
    griddep_launch_dependents();
    if (aborted && tid == 0) {
        // the copies that are still in flight: the row before's stage was not refilled
        const int64_t from = j > 0 ? j - 1 : 0;
        for (int64_t i = j; i < (from + S < nrows ? from + S : nrows); ++i)
            mbar_wait_bounded(smem_u32(&full[i % S]), static_cast<uint32_t>((i / S) & 1), a.err, 1u << 16);
    }
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
template <int DT, int MODE>
static const void* bwd_rows_for(int lanes, int octets) {
#define RMSNORM_ADD_BWD(G, KB) \
    if (lanes == G && octets == KB) return reinterpret_cast<const void*>(&add_bwd_rows<DT, MODE, G, KB>);
    RMSNORM_ADD_BWD(8, 1)
    RMSNORM_ADD_BWD(8, 2)
    RMSNORM_ADD_BWD(32, 1)
    RMSNORM_ADD_BWD(32, 2)
    if constexpr (MODE != kRowsOnePhase) {  // blocks take such rows from 65 octets on
        RMSNORM_ADD_BWD(32, 4)
    }
    RMSNORM_ADD_BWD(0, 2)
    RMSNORM_ADD_BWD(0, 4)
    if constexpr (MODE != kRowsAligned) {
        RMSNORM_ADD_BWD(0, 5)
    }
#undef RMSNORM_ADD_BWD
    return nullptr;
}
template <int DT, bool AL, bool DROP>
static const void* bwd_ring_for(int octets) {
    switch (octets) {
    case 2: return reinterpret_cast<const void*>(&add_bwd_ring<DT, AL, 2, DROP>);
    case 3: return reinterpret_cast<const void*>(&add_bwd_ring<DT, AL, 3, DROP>);
    case 4: return reinterpret_cast<const void*>(&add_bwd_ring<DT, AL, 4, DROP>);
    default: return nullptr;
    }
}
template <int DT>
static const void* bwd_dtype(const AddPlan& p) {
    if (!p.ring) {
        switch (p.mode) {
        case kRowsAligned: return bwd_rows_for<DT, kRowsAligned>(p.lanes, p.octets);
        case kRowsOnePhase: return bwd_rows_for<DT, kRowsOnePhase>(p.lanes, p.octets);
        default: return bwd_rows_for<DT, kRowsAny>(p.lanes, p.octets);
        }
    }
    if (p.drop) return p.mode == kRowsAligned ? bwd_ring_for<DT, true, true>(p.octets) : bwd_ring_for<DT, false, true>(p.octets);
    return p.mode == kRowsAligned ? bwd_ring_for<DT, true, false>(p.octets) : bwd_ring_for<DT, false, false>(p.octets);
}

const void* add_bwd_kernel(const AddPlan& p) {
    switch (p.dtype) {
    case kF32: return bwd_dtype<kF32>(p);
    case kF16: return bwd_dtype<kF16>(p);
    case kBF16: return bwd_dtype<kBF16>(p);
    default: return nullptr;
    }
}

}  // namespace rmsnorm
