// rope.cu -- RMSNorm of attention heads and the rotation of their first R entries by
// the token's position, forward and backward.
//
// Per head row x of D entries: n = x * r with r = 1 / sqrt(sum(x^2) / D + eps),
// z = n * g (z = x without a weight: the rotation alone), and for each pair (a, b)
// of the first R entries, with the angle t = position * inv_freq:
//     out_a = z_a * cos t - z_b * sin t,   out_b = z_b * cos t + z_a * sin t
// (cos and sin times mscale); the entries from R on are z. Pairs are (2i, 2i + 1)
// (interleaved) or (i, i + R / 2). The backward turns the cotangent back (the same
// with -t), v, and then u = v * g, dx = r * (u - n * (sum(u * n) / D)),
// dgamma = sum over tokens and heads of v * n. It recomputes r from x, which it
// reads anyway: the forward stores nothing for it.
//
// Angles: position * inv_freq loses the angle in fp32 (at position 10^6 by 0.06
// radians) and fp64 is slow on this GPU, but only the fraction of a turn matters.
// Each inv_freq becomes a 64-bit fixed-point number of turns per position; its
// product with the integer position, modulo 2^64, is the fraction exactly reduced.
#include "fused.h"
#include "launch.h"
#include "octet.cuh"

namespace rmsnorm {

// f radians as turns in units of 2^-64, modulo one turn: f = m * 2^(e - 63) with a
// 64-bit mantissa m, and hi64(m * 2^64 * 2 / pi) * 2^(e - 1) = f / (2 pi) * 2^64.
__device__ __forceinline__ uint64_t turns_per_position(double f) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(f));
    const int e = static_cast<int>((b >> 52) & 0x7ff) - 1023;
    const uint64_t m = (b << 11) | 0x8000000000000000ull;
    const uint64_t p = __umul64hi(m, 0xA2F9836E4E44152Aull);  // 2 / pi * 2^64
    uint64_t t = 0;  // also for 0 and subnormal f
    if (e <= 1) {
        if (e > -63) t = p >> (1 - e);
    } else if (e < 65) {
        t = p << (e - 1);
    }
    return (b >> 63) ? 0ull - t : t;
}

__device__ __forceinline__ void turn_at(uint64_t per_position, int64_t pos, float mscale, float& c, float& s) {
    const uint64_t phase = per_position * static_cast<uint64_t>(pos);
    const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
    sincospif(half_turns, &s, &c);
    c *= mscale;
    s *= mscale;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The heads of a set among the heads [lo, hi) of all sets, the set's first being
// head `at` of all.
__device__ __forceinline__ void heads_of(const RopeSet& s, int at, int lo, int hi, int& from, int& to) {
    from = lo > at ? lo - at : 0;
    to = hi - at < s.heads ? hi - at : s.heads;
}

// The 16 entries of a head row that a lane owns: two octets, eight pairs. Pairs
// are neighbours in an octet (INTER) or the same entry of both octets.
template <bool INTER>
__device__ __forceinline__ void lane_octets(int li, int D, int R, int& a, int& b) {
    const int n = D / 8;
    if (INTER) {
        a = 2 * li;
        b = a + 1;
    } else if (li < R / 16) {
        a = li;
        b = li + R / 16;
    } else {
        a = R / 8 + 2 * (li - R / 16);
        b = a + 1;
    }
    if (a >= n) a = -1;
    if (b >= n) b = -1;
}

template <bool INTER>
__device__ __forceinline__ void rotate(float (&f)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float& p = f[INTER ? 2 * k : k];
        float& q = f[INTER ? 2 * k + 1 : k + 8];
        const float x = p, y = q;
        p = x * c[k] - y * s[k];
        q = y * c[k] + x * s[k];
    }
}

template <int DT>
__device__ __forceinline__ void load16(const char* row, int a, int b, bool live, uint32_t (&w)[2][Oct<DT>::kWords]) {
#pragma unroll
    for (int i = 0; i < Oct<DT>::kWords; ++i) w[0][i] = w[1][i] = 0u;
    if (live && a >= 0) octet_load<DT, true>(row + a * Oct<DT>::kBytes, 0, 8, w[0]);
    if (live && b >= 0) octet_load<DT, true>(row + b * Oct<DT>::kBytes, 0, 8, w[1]);
}
template <int DT>
__device__ __forceinline__ void unpack16(const uint32_t (&w)[2][Oct<DT>::kWords], float (&f)[16]) {
    Oct<DT>::unpack(w[0], *reinterpret_cast<float(*)[8]>(&f[0]));
    Oct<DT>::unpack(w[1], *reinterpret_cast<float(*)[8]>(&f[8]));
}
template <int DT>
__device__ __forceinline__ void store16(char* row, int a, int b, const float (&f)[16]) {
    uint32_t w[Oct<DT>::kWords];
    Oct<DT>::pack(*reinterpret_cast<const float(*)[8]>(&f[0]), w);
    octet_store<Elem<DT>::kBytes, Oct<DT>::kWords, true>(row + a * Oct<DT>::kBytes, w, a >= 0 ? Oct<DT>::kBytes : 0, false,
                                                         false);
    Oct<DT>::pack(*reinterpret_cast<const float(*)[8]>(&f[8]), w);
    octet_store<Elem<DT>::kBytes, Oct<DT>::kWords, true>(row + b * Oct<DT>::kBytes, w, b >= 0 ? Oct<DT>::kBytes : 0, false,
                                                         false);
}

// Rows of whole octets: a group of `lanes` lanes (4 to 32) takes a chunk of a
// token's heads, its cosines and sines computed once and kept in registers; the
// loads of several heads go out together.
template <int DT, bool INTER>
__global__ void __launch_bounds__(kFusedGroupThreads) rope_fwd_octets(const RopeArgs a, int lanes) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    constexpr int BATCH = DT == kF32 ? 2 : 4;
    const int li = threadIdx.x % lanes;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    griddep_wait();
    const bool live = item < a.T * a.nchunk;
    const int64_t token = live ? item / a.nchunk : 0;
    const int lo = live ? static_cast<int>(item % a.nchunk) * a.chunk : 0;
    const int hi = live ? min(lo + a.chunk, a.heads) : 0;
    int oa, ob;
    lane_octets<INTER>(li, a.D, a.R, oa, ob);
    float c[8], s[8];
    const int64_t pos = a.pos[token];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        c[k] = 1.f;
        s[k] = 0.f;
        if (8 * li + k < a.R / 2) turn_at(turns_per_position(a.inv_freq[8 * li + k]), pos, a.mscale, c[k], s[k]);
    }
    const float inv_d = 1.0f / static_cast<float>(a.D);
    int at = 0;
    for (int i = 0; i < a.nsets; ++i) {
        const RopeSet& set = a.set[i];
        int from, to;
        heads_of(set, at, lo, hi, from, to);
        at += set.heads;
        // every lane of the warp runs the longest of its groups' counts (the sums
        // see the whole warp); all groups but a token's last have the same
        const int n = to > from ? to - from : 0;
        const int most = static_cast<int>(warp_allmax(static_cast<uint32_t>(n)));
        uint32_t gw[2][W];
        load16<DT>(static_cast<const char*>(set.gamma), oa, ob, set.gamma != nullptr, gw);
        const char* xb = static_cast<const char*>(set.x) + (token * set.x_token + from * set.x_head) * EB;
        char* yb = static_cast<char*>(set.y) + (token * set.y_token + from * set.y_head) * EB;
        for (int h = 0; h < most; h += BATCH) {
            uint32_t xw[BATCH][2][W];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) load16<DT>(xb + (h + j) * set.x_head * EB, oa, ob, h + j < n, xw[j]);
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                float f[16];
                unpack16<DT>(xw[j], f);
                if (set.gamma) {
                    float g[16], ss = 0.f;
                    unpack16<DT>(gw, g);
#pragma unroll
                    for (int e = 0; e < 16; ++e) ss = fmaf(f[e], f[e], ss);
                    const float r = 1.0f / sqrtf(lanes_sum(ss, lanes) * inv_d + a.eps);
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = (f[e] * r) * (g[e] + a.one);
                }
                rotate<INTER>(f, c, s);
                if (h + j < n) store16<DT>(yb + (h + j) * set.y_head * EB, oa, ob, f);
            }
        }
    }
    griddep_launch_dependents();
}

// The backward on the same rows: persistent, so that a lane, which owns the same
// columns of every head, adds its share of dgamma up in registers; each block
// writes one row of partials per set for the fixed-order column reduce.
template <int DT, bool INTER>
__global__ void __launch_bounds__(kFusedGroupThreads) rope_bwd_octets(const RopeArgs a, int lanes) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    extern __shared__ float sums[];  // [groups of the block][D]
    const int li = threadIdx.x % lanes;
    const int groups = blockDim.x / lanes;
    const int group = threadIdx.x / lanes;
    griddep_wait();
    int oa, ob;
    lane_octets<INTER>(li, a.D, a.R, oa, ob);
    uint64_t turn[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) turn[k] = 8 * li + k < a.R / 2 ? turns_per_position(a.inv_freq[8 * li + k]) : 0ull;
    float acc[kRopeMaxSets][16];
#pragma unroll
    for (int i = 0; i < kRopeMaxSets; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    const int64_t items = a.T * a.nchunk;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < items;
         base += static_cast<int64_t>(gridDim.x) * groups) {
        const int64_t item = base + group;
        const bool live = item < items;
        const int64_t token = live ? item / a.nchunk : 0;
        const int lo = live ? static_cast<int>(item % a.nchunk) * a.chunk : 0;
        const int hi = live ? min(lo + a.chunk, a.heads) : 0;
        const int64_t pos = a.pos[token];
        float c[8], s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            c[k] = 1.f;
            s[k] = 0.f;
            if (8 * li + k < a.R / 2) {
                turn_at(turn[k], pos, a.mscale, c[k], s[k]);
                s[k] = -s[k];
            }
        }
        int at = 0;
#pragma unroll
        for (int i = 0; i < kRopeMaxSets; ++i) {
            if (i >= a.nsets) break;
            const RopeSet& set = a.set[i];
            int from, to;
            heads_of(set, at, lo, hi, from, to);
            at += set.heads;
            const int n = to > from ? to - from : 0;
            const int most = static_cast<int>(warp_allmax(static_cast<uint32_t>(n)));
            uint32_t gw[2][W];
            load16<DT>(static_cast<const char*>(set.gamma), oa, ob, set.gamma != nullptr, gw);
            const char* db = static_cast<const char*>(set.dy) + (token * set.dy_token + from * set.dy_head) * EB;
            const char* xb = static_cast<const char*>(set.x) + (token * set.x_token + from * set.x_head) * EB;
            char* yb = static_cast<char*>(set.y) + (token * set.y_token + from * set.y_head) * EB;
            for (int h = 0; h < most; ++h) {
                uint32_t dw[2][W], xw[2][W];
                load16<DT>(db + h * set.dy_head * EB, oa, ob, h < n, dw);
                load16<DT>(xb + h * set.x_head * EB, oa, ob, h < n && set.gamma != nullptr, xw);
                float v[16];
                unpack16<DT>(dw, v);
                rotate<INTER>(v, c, s);
                if (set.gamma) {
                    float x[16], g[16], ss = 0.f, q = 0.f;
                    unpack16<DT>(xw, x);
                    unpack16<DT>(gw, g);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        ss = fmaf(x[e], x[e], ss);
                        q = fmaf(v[e] * (g[e] + a.one), x[e], q);
                    }
                    const float r = 1.0f / sqrtf(lanes_sum(ss, lanes) * inv_d + a.eps);
                    const float m = lanes_sum(q, lanes) * inv_d * r;  // mean(u * n)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float nv = x[e] * r;
                        acc[i][e] = fmaf(v[e], nv, acc[i][e]);
                        v[e] = r * (v[e] * (g[e] + a.one) - nv * m);
                    }
                }
                if (h < n) store16<DT>(yb + h * set.y_head * EB, oa, ob, v);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRopeMaxSets; ++i) {
        if (i >= a.nsets) break;
        if (!a.set[i].gamma) continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (oa >= 0) sums[group * a.D + 8 * oa + e] = acc[i][e];
            if (ob >= 0) sums[group * a.D + 8 * ob + e] = acc[i][8 + e];
        }
        __syncthreads();
        float* out = a.ws + (i * a.units + blockIdx.x) * a.ldws;
        for (int col = threadIdx.x; col < a.D; col += blockDim.x) {
            float t = sums[col];
            for (int k = 1; k < groups; ++k) t += sums[k * a.D + col];
            out[col] = t;
        }
    }
    griddep_launch_dependents();
}

// Any D, R and alignment: a warp takes a chunk of a token's heads, a lane the pairs
// li, li + 32, ... (PK of them at most), loaded and stored entry by entry. The
// entries from R on are paired as neighbours and not turned.
template <int PK>
__device__ __forceinline__ void lane_pairs(int li, const RopeArgs& a, bool inter, int (&ca)[PK], int (&cb)[PK]) {
    const int half = a.R / 2;
#pragma unroll
    for (int k = 0; k < PK; ++k) {
        const int i = li + 32 * k;
        if (i < half) {
            ca[k] = inter ? 2 * i : i;
            cb[k] = inter ? 2 * i + 1 : i + half;
        } else {
            ca[k] = a.R + 2 * (i - half);
            cb[k] = ca[k] + 1;
        }
        if (ca[k] >= a.D) ca[k] = -1;
        if (cb[k] >= a.D) cb[k] = -1;
    }
}

// Plain (not read-only-cache) loads: an output may be its input.
template <int DT> __device__ __forceinline__ float entry(const char* p, int64_t i) {
    if constexpr (DT == kF32) return reinterpret_cast<const float*>(p)[i];
    else if constexpr (DT == kF16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    else return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

template <int DT, int PK, bool BWD>
__global__ void __launch_bounds__(kFusedGroupThreads) rope_pairs(const RopeArgs a, int inter) {
    constexpr int EB = Elem<DT>::kBytes;
    extern __shared__ float sums[];  // backward: [warps of the block][D]
    const int li = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    griddep_wait();
    int ca[PK], cb[PK];
    lane_pairs<PK>(li, a, inter != 0, ca, cb);
    float acc[BWD ? kRopeMaxSets : 1][2 * PK];
#pragma unroll
    for (int i = 0; i < (BWD ? kRopeMaxSets : 1); ++i)
#pragma unroll
        for (int k = 0; k < 2 * PK; ++k) acc[i][k] = 0.f;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    const int64_t items = a.T * a.nchunk;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * warps + warp; item < items;
         item += static_cast<int64_t>(gridDim.x) * warps) {
        const int64_t token = item / a.nchunk;
        const int lo = static_cast<int>(item % a.nchunk) * a.chunk;
        const int hi = min(lo + a.chunk, a.heads);
        const int64_t pos = a.pos[token];
        float c[PK], s[PK];
#pragma unroll
        for (int k = 0; k < PK; ++k) {
            c[k] = 1.f;
            s[k] = 0.f;
            if (li + 32 * k < a.R / 2) {
                turn_at(turns_per_position(a.inv_freq[li + 32 * k]), pos, a.mscale, c[k], s[k]);
                if (BWD) s[k] = -s[k];
            }
        }
        int at = 0;
#pragma unroll
        for (int i = 0; i < kRopeMaxSets; ++i) {
            if (i >= a.nsets) break;
            const RopeSet& set = a.set[i];
            int from, to;
            heads_of(set, at, lo, hi, from, to);
            at += set.heads;
            const char* gb = static_cast<const char*>(set.gamma);
            for (int h = from; h < to; ++h) {
                const char* xr = static_cast<const char*>(set.x) + (token * set.x_token + h * set.x_head) * EB;
                const char* dr = static_cast<const char*>(set.dy) + (token * set.dy_token + h * set.dy_head) * EB;
                char* yr = static_cast<char*>(set.y) + (token * set.y_token + h * set.y_head) * EB;
                float x[2 * PK], v[2 * PK], g[2 * PK];
                float ss = 0.f, q = 0.f;
#pragma unroll
                for (int k = 0; k < PK; ++k) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int col = e ? cb[k] : ca[k];
                        const int j = 2 * k + e;
                        x[j] = v[j] = 0.f;
                        g[j] = 1.f;
                        if (col >= 0) {
                            if (!BWD || gb) x[j] = entry<DT>(xr, col);
                            if (BWD) v[j] = entry<DT>(dr, col);
                            if (gb) g[j] = entry<DT>(gb, col) + a.one;
                        }
                    }
                    if (BWD) {
                        const float p = v[2 * k], z = v[2 * k + 1];
                        v[2 * k] = p * c[k] - z * s[k];
                        v[2 * k + 1] = z * c[k] + p * s[k];
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 2 * k + e;
                        ss = fmaf(x[j], x[j], ss);
                        q = fmaf(v[j] * g[j], x[j], q);
                    }
                }
                float r = 1.f, m = 0.f;
                if (gb) {
                    r = 1.0f / sqrtf(warp_allsum(ss) * inv_d + a.eps);
                    if (BWD) m = warp_allsum(q) * inv_d * r;
                }
#pragma unroll
                for (int k = 0; k < PK; ++k) {
                    float o0, o1;
                    if (BWD) {
                        o0 = v[2 * k];
                        o1 = v[2 * k + 1];
                        if (gb) {
                            const float n0 = x[2 * k] * r, n1 = x[2 * k + 1] * r;
                            acc[BWD ? i : 0][2 * k] = fmaf(o0, n0, acc[BWD ? i : 0][2 * k]);
                            acc[BWD ? i : 0][2 * k + 1] = fmaf(o1, n1, acc[BWD ? i : 0][2 * k + 1]);
                            o0 = r * (o0 * g[2 * k] - n0 * m);
                            o1 = r * (o1 * g[2 * k + 1] - n1 * m);
                        }
                    } else {
                        const float z0 = (x[2 * k] * r) * g[2 * k], z1 = (x[2 * k + 1] * r) * g[2 * k + 1];
                        o0 = z0 * c[k] - z1 * s[k];
                        o1 = z1 * c[k] + z0 * s[k];
                    }
                    if (ca[k] >= 0) Elem<DT>::st(yr, ca[k], o0);
                    if (cb[k] >= 0) Elem<DT>::st(yr, cb[k], o1);
                }
            }
        }
    }
    if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < kRopeMaxSets; ++i) {
            if (i >= a.nsets) break;
            if (!a.set[i].gamma) continue;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < PK; ++k) {
                if (ca[k] >= 0) sums[warp * a.D + ca[k]] = acc[i][2 * k];
                if (cb[k] >= 0) sums[warp * a.D + cb[k]] = acc[i][2 * k + 1];
            }
            __syncthreads();
            float* out = a.ws + (i * a.units + blockIdx.x) * a.ldws;
            for (int col = threadIdx.x; col < a.D; col += blockDim.x) {
                float t = sums[col];
                for (int k = 1; k < warps; ++k) t += sums[k * a.D + col];
                out[col] = t;
            }
        }
    }
    griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// dispatch: `lanes` is the lanes per row of the octet kernels, the pairs per lane of
// the others
// ---------------------------------------------------------------------------
template <int DT>
static const void* rope_kernel_for(const RopePlan& p, bool bwd) {
    if (p.aligned) {
        if (p.interleaved)
            return bwd ? reinterpret_cast<const void*>(&rope_bwd_octets<DT, true>)
                       : reinterpret_cast<const void*>(&rope_fwd_octets<DT, true>);
        return bwd ? reinterpret_cast<const void*>(&rope_bwd_octets<DT, false>)
                   : reinterpret_cast<const void*>(&rope_fwd_octets<DT, false>);
    }
    if (p.lanes <= 2)
        return bwd ? reinterpret_cast<const void*>(&rope_pairs<DT, 2, true>)
                   : reinterpret_cast<const void*>(&rope_pairs<DT, 2, false>);
    return bwd ? reinterpret_cast<const void*>(&rope_pairs<DT, 8, true>)
               : reinterpret_cast<const void*>(&rope_pairs<DT, 8, false>);
}

const void* rope_kernel(const RopePlan& p, bool bwd) {
    switch (p.dtype) {
    case kF32: return rope_kernel_for<kF32>(p, bwd);
    case kF16: return rope_kernel_for<kF16>(p, bwd);
    case kBF16: return rope_kernel_for<kBF16>(p, bwd);
    default: return nullptr;
    }
}

}  // namespace rmsnorm
