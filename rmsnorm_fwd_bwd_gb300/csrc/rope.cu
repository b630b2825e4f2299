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
// product with the integer position, modulo 2^64, is the fraction exactly reduced. All its
// bits count in what is left of a quarter turn, the fp32 angle of the series.
//
// Bound by HBM: the heads in and out (backward: dy and x in, dx out). Measured on GB300 (a
// device copy moves 6.77 TB/s): forward 32768 tokens x 40 heads x 128 bf16 104 us (6.4
// TB/s; 138 us with the sines by sincospif and all heads of a token by one group, 125 us
// with two heads in flight a lane instead of four), fp32 16384 x 40 x 128 97 us (6.9
// TB/s); backward 16384 x 20 x 256 bf16 94 us (5.35 TB/s, bound by latency at 12 warps an
// SM: its sums and weight hold the registers). 64 tokens: 2.2 us a call in a graph. Halves
// that do not meet octet by octet swap partners through shared memory (rope_fwd_swap); head
// rows off 16 bytes or of no whole octets go entry by entry, at 19-60% of the copy's rate.
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

// The turn's fraction at a position, in units of 2^-64 (a signed half turn either way).
__device__ __forceinline__ int64_t phase_at(uint64_t per_position, int64_t pos) {
    return static_cast<int64_t>(per_position * static_cast<uint64_t>(pos));
}

// What is left of a phase when the nearest quarter turn is taken off, as upper * 2^32 + lower,
// each rounded to fp32: small angles, of slow pairs at near positions, have all its bits too
// (the upper word alone is off by 1.5e-4 of an angle of 10^-5 radians; one conversion
// from 64 bits cost the forward 2.6%, two from 32 nothing). q: the phase's upper
// word, an eighth of a turn on.
__device__ __forceinline__ void quarter_rest(int64_t p, uint32_t& q, float& upper, float& lower) {
    const int32_t low = static_cast<int32_t>(p);  // below 0 it borrows from the upper word
    q = static_cast<uint32_t>(static_cast<uint64_t>(p) >> 32) + 0x20000000u;
    upper = static_cast<float>(static_cast<int32_t>(q & 0x3fffffffu) - 0x20000000 - (low >> 31));
    lower = static_cast<float>(low);
}

// cos and sin, times m, of two angles given as phases. The nearest quarter turn is taken
// off, and the rest, below pi / 4, goes through the Taylor series: sin to t^9 (the next
// term is below 2^-28 there), cos to t^10 (below 2^-32), both angles in one packed
// instruction. About half the instructions of two sincospif calls.
__device__ __forceinline__ void turn_pair(int64_t p0, int64_t p1, float m0, float m1, uint64_t& c, uint64_t& s) {
    uint32_t q0, q1;
    auto both = [](float v) { return f2_pack(v, v); };
    float u0, u1, l0, l1;
    quarter_rest(p0, q0, u0, l0);
    quarter_rest(p1, q1, u1, l1);
    // in radians: 2 pi / 2^32 and 2 pi / 2^64
    const uint64_t t = f2_fma(f2_pack(u0, u1), both(1.4629180792671596e-9f),
                              f2_mul(f2_pack(l0, l1), both(3.4061215800865545e-19f)));
    const uint64_t z = f2_mul(t, t);
    uint64_t p = f2_fma(z, both(1.f / 362880), both(-1.f / 5040));
    p = f2_fma(p, z, both(1.f / 120));
    p = f2_fma(p, z, both(-1.f / 6));
    const uint64_t sn = f2_fma(f2_mul(t, z), p, t);
    p = f2_fma(z, both(-1.f / 3628800), both(1.f / 40320));
    p = f2_fma(p, z, both(-1.f / 720));
    p = f2_fma(p, z, both(1.f / 24));
    p = f2_fma(p, z, both(-1.f / 2));
    const uint64_t cs = f2_fma(p, z, both(1.f));
    float s0, s1, c0, c1;
    f2_unpack(sn, s0, s1);
    f2_unpack(cs, c0, c1);
    // quarter turns: 1 swaps (cos, sin) to (-sin, cos), 2 turns both signs
    auto turned = [](uint32_t q, float& a, float& b) {
        const float x = (q & 0x40000000u) ? b : a, y = (q & 0x40000000u) ? a : b;
        a = __uint_as_float(__float_as_uint(x) ^ ((q + 0x40000000u) & 0x80000000u));
        b = __uint_as_float(__float_as_uint(y) ^ (q & 0x80000000u));
    };
    turned(q0, c0, s0);
    turned(q1, c1, s1);
    const uint64_t m = f2_pack(m0, m1);
    c = f2_mul(f2_pack(c0, c1), m);
    s = f2_mul(f2_pack(s0, s1), m);
}

// item = token * n + chunk, by a 32-bit division where it fits.
__device__ __forceinline__ int64_t split_item(int64_t item, int n, int& chunk) {
    if (item < (int64_t(1) << 32)) {
        const uint32_t t = static_cast<uint32_t>(item) / static_cast<uint32_t>(n);
        chunk = static_cast<int>(static_cast<uint32_t>(item) - t * static_cast<uint32_t>(n));
        return t;
    }
    const int64_t t = item / n;
    chunk = static_cast<int>(item - t * n);
    return t;
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

// The octets as the pairs' first entries p and second entries q, packed two pairs to a
// word; and back.
template <int DT, bool INTER>
__device__ __forceinline__ void to_pairs(const uint32_t (&w)[2][Oct<DT>::kWords], uint64_t (&p)[4], uint64_t (&q)[4]) {
    float f[16];
    Oct<DT>::unpack(w[0], *reinterpret_cast<float(*)[8]>(&f[0]));
    Oct<DT>::unpack(w[1], *reinterpret_cast<float(*)[8]>(&f[8]));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = INTER ? f2_pack(f[4 * i], f[4 * i + 2]) : f2_pack(f[2 * i], f[2 * i + 1]);
        q[i] = INTER ? f2_pack(f[4 * i + 1], f[4 * i + 3]) : f2_pack(f[8 + 2 * i], f[9 + 2 * i]);
    }
}
template <int DT, bool INTER>
__device__ __forceinline__ void store_pairs(char* row, int a, int b, const uint64_t (&p)[4], const uint64_t (&q)[4]) {
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f2_unpack(p[i], INTER ? f[4 * i] : f[2 * i], INTER ? f[4 * i + 2] : f[2 * i + 1]);
        f2_unpack(q[i], INTER ? f[4 * i + 1] : f[8 + 2 * i], INTER ? f[4 * i + 3] : f[9 + 2 * i]);
    }
    uint32_t w[Oct<DT>::kWords];
    constexpr int EB = Elem<DT>::kBytes, B = Oct<DT>::kBytes;
    Oct<DT>::pack(*reinterpret_cast<const float(*)[8]>(&f[0]), w);
    octet_store<EB, Oct<DT>::kWords, true>(row + a * B, w, a >= 0 ? B : 0, false, false);
    Oct<DT>::pack(*reinterpret_cast<const float(*)[8]>(&f[8]), w);
    octet_store<EB, Oct<DT>::kWords, true>(row + b * B, w, b >= 0 ? B : 0, false, false);
}

template <int DT>
__device__ __forceinline__ void load16(const char* row, int a, int b, bool live, uint32_t (&w)[2][Oct<DT>::kWords]) {
#pragma unroll
    for (int i = 0; i < Oct<DT>::kWords; ++i) w[0][i] = w[1][i] = 0u;
    if (live && a >= 0) octet_load<DT, true>(row + a * Oct<DT>::kBytes, 0, 8, w[0]);
    if (live && b >= 0) octet_load<DT, true>(row + b * Oct<DT>::kBytes, 0, 8, w[1]);
}

// A lane's gains g or 1 + g (1 without a weight), as pairs.
template <int DT, bool INTER>
__device__ __forceinline__ void load_gains(const RopeSet& set, float one, int oa, int ob, uint64_t (&gp)[4], uint64_t (&gq)[4]) {
    uint32_t w[2][Oct<DT>::kWords];
    load16<DT>(static_cast<const char*>(set.gamma), oa, ob, set.gamma != nullptr, w);
    to_pairs<DT, INTER>(w, gp, gq);
    const float add = set.gamma ? one : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        gp[i] = f2_add(gp[i], f2_pack(add, add));
        gq[i] = f2_add(gq[i], f2_pack(add, add));
    }
}

// The turns per position of a row's pairs, in shared memory: lane li's eight at [k][li],
// 0 from entry R on (to be followed by a block barrier).
struct Turns {
    uint64_t at[8][32];
    __device__ __forceinline__ void fill(const RopeArgs& a, int lanes) {
        for (int i = threadIdx.x; i < 8 * lanes; i += blockDim.x) {
            const int li = i / 8, k = i % 8;
            at[k][li] = i < a.R / 2 ? turns_per_position(a.inv_freq[i]) : 0ull;
        }
    }
    // cos and sin (times mscale) of a lane's pairs at a position; 1 and 0 from entry R on
    __device__ __forceinline__ void of_lane(const RopeArgs& a, int li, int64_t pos, uint64_t (&c)[4], uint64_t (&s)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 8 * li + 2 * i;
            turn_pair(phase_at(at[2 * i][li], pos), phase_at(at[2 * i + 1][li], pos), k < a.R / 2 ? a.mscale : 1.f,
                      k + 1 < a.R / 2 ? a.mscale : 1.f, c[i], s[i]);
        }
    }
};

__device__ __forceinline__ uint64_t f2_neg(uint64_t v) { return v ^ 0x8000000080000000ull; }

// How many of a lane's eight pairs are rotated, the first ones: all or none of them but
// where neighbours are paired.
__device__ __forceinline__ int rotated_pairs(const RopeArgs& a, int li) { return max(0, min(8, a.R / 2 - 8 * li)); }

// Plain (not read-only-cache) loads: an output may be its input.
template <int DT> __device__ __forceinline__ float entry(const char* p, int64_t i) {
    if constexpr (DT == kF32) return reinterpret_cast<const float*>(p)[i];
    else if constexpr (DT == kF16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    else return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// The lane's pairs (p, q) to p * cp + q * sp and q * cq + p * sq.
__device__ __forceinline__ void turn_pairs(uint64_t (&p)[4], uint64_t (&q)[4], const uint64_t (&cp)[4], const uint64_t (&sp)[4],
                                           const uint64_t (&cq)[4], const uint64_t (&sq)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t x = p[k], y = q[k];
        p[k] = f2_fma(x, cp[k], f2_mul(y, sp[k]));
        q[k] = f2_fma(y, cq[k], f2_mul(x, sq[k]));
    }
}

// The same for the first `rotated` pairs, the others to p * cp and q * cq.
template <bool INTER>
__device__ __forceinline__ void turn_first_pairs(int rotated, uint64_t (&p)[4], uint64_t (&q)[4], const uint64_t (&cp)[4],
                                                 const uint64_t (&sp)[4], const uint64_t (&cq)[4], const uint64_t (&sq)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t x = p[k], y = q[k];
        const uint64_t keep = (2 * k < rotated ? 0xffffffffull : 0ull) |
                              ((INTER ? 2 * k + 1 : 2 * k) < rotated ? 0xffffffffull << 32 : 0ull);
        p[k] = f2_fma(x, cp[k], f2_mul(y & keep, sp[k]));
        q[k] = f2_fma(y, cq[k], f2_mul(x & keep, sq[k]));
    }
}

// The same again from the row in memory, entry by entry, with few registers. An infinity or
// a NaN behind the rotated entries times a sine of 0 would be a NaN in its neighbour: a
// row where that happened is done again, but for the fp32 backward, whose registers have no
// room for it and whose entries are masked. (bf16 forward, half of 128 entries
// rotated: 101.4 us without, 102.7 so, 114 with two ways for every row; fp32 backward 81.5
// without, 90.4 masked, 97-107 done again, 104 masked behind a branch on R < D.)
template <int DT, bool INTER>
__device__ __forceinline__ void turn_again(const char* row, int oa, int ob, int rotated, uint64_t (&p)[4], uint64_t (&q)[4],
                                           const uint64_t (&cp)[4], const uint64_t (&sp)[4], const uint64_t (&cq)[4],
                                           const uint64_t (&sq)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a[2], b[2], ca[2], sa[2], cb[2], sb[2];
        f2_unpack(cp[k], ca[0], ca[1]);
        f2_unpack(sp[k], sa[0], sa[1]);
        f2_unpack(cq[k], cb[0], cb[1]);
        f2_unpack(sq[k], sb[0], sb[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 2 * k + h;
            const int o = INTER && i >= 4 ? ob : oa, o2 = INTER ? o : ob;
            const float x = o >= 0 ? entry<DT>(row, 8 * o + (INTER ? 2 * (i & 3) : i)) : 0.f;
            const float y = o2 >= 0 ? entry<DT>(row, 8 * o2 + (INTER ? 2 * (i & 3) + 1 : i)) : 0.f;
            a[h] = i < rotated ? fmaf(x, ca[h], y * sa[h]) : x * ca[h];
            b[h] = i < rotated ? fmaf(y, cb[h], x * sb[h]) : y * cb[h];
        }
        p[k] = f2_pack(a[0], a[1]);
        q[k] = f2_pack(b[0], b[1]);
    }
}

__device__ __forceinline__ float f2_sum(uint64_t v) {
    float a, b;
    f2_unpack(v, a, b);
    return a + b;
}

// Rows of whole octets: a group of L lanes (4 to 32, the fewest that hold a row at 16
// entries each) takes up to BATCH heads of a token; neighbouring groups take
// neighbouring heads. The heads' loads go out first, and the cosines and sines are
// computed while they are under way and folded into the weight:
// out_a = r * (x_a * (g_a cos) - x_b * (g_b sin)), out_b = r * (x_b * (g_b cos) + x_a *
// (g_a sin)).
template <int DT, bool INTER, int L>
__global__ void __maxnreg__(96) rope_fwd_octets(const RopeArgs a) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    constexpr int BATCH = rope_fwd_batch(DT);
    __shared__ Turns turns;
    const int li = threadIdx.x % L;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x / L) + threadIdx.x / L;
    griddep_wait();
    const bool live = item < a.T * a.nchunk;
    int chunk;
    const int64_t token = split_item(live ? item : 0, a.nchunk, chunk);
    const int which = chunk >= a.chunks0 ? 1 : 0;
    if (which) chunk -= a.chunks0;
    const RopeSet& set = a.set[which];
    const int from = chunk * a.chunk;
    const int n = live ? min(a.chunk, set.heads - from) : 0;
    int oa, ob;
    lane_octets<INTER>(li, a.D, a.R, oa, ob);
    const int rotated = rotated_pairs(a, li);
    const char* xb = static_cast<const char*>(set.x) + (token * set.x_token + from * set.x_head) * EB;
    char* yb = static_cast<char*>(set.y) + (token * set.y_token + from * set.y_head) * EB;
    const int64_t x_step = set.x_head * EB, y_step = set.y_head * EB;
    uint32_t xw[BATCH][2][W];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) load16<DT>(xb + j * x_step, oa, ob, j < n, xw[j]);
    uint64_t pc[4], ps[4], qc[4], qs[4];
    load_gains<DT, INTER>(set, a.one, oa, ob, pc, qc);
    const int64_t pos = a.pos[token];
    turns.fill(a, L);
    __syncthreads();
    {
        uint64_t c[4], s[4];
        turns.of_lane(a, li, pos, c, s);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            ps[k] = f2_mul(pc[k], s[k]);
            pc[k] = f2_mul(pc[k], c[k]);
            qs[k] = f2_neg(f2_mul(qc[k], s[k]));
            qc[k] = f2_mul(qc[k], c[k]);
        }
    }
    // Rows with an infinity or a NaN are turned again, as their sum of squares tells; all rows are
    // where a sine of 0 met such a gain behind the rotated entries (bf16, half of 128 rotated:
    // 103.7 us without, 104.6 so, 104.9 with masked products).
    uint64_t sines = f2_add(ps[0], qs[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) sines = f2_add(sines, f2_add(ps[k], qs[k]));
    const float all = f2_sum(sines);
    const float finite = all == all ? __int_as_float(0x7f800000) : 0.f;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    // chunk is the same everywhere: the whole warp goes round as often (the sums see it)
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
        if (j >= a.chunk) break;
        uint64_t p[4], q[4];
        to_pairs<DT, INTER>(xw[j], p, q);
        uint64_t ss = f2_mul(p[0], p[0]);
#pragma unroll
        for (int k = 1; k < 4; ++k) ss = f2_fma(p[k], p[k], ss);
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = f2_fma(q[k], q[k], ss);
        const float sum = row_sum<L>(f2_sum(ss), nullptr);
        const float r = set.gamma ? row_rsqrt(sum, inv_d, a.eps) : 1.f;
        const uint64_t r2 = f2_pack(r, r);
        turn_pairs(p, q, pc, qs, qc, ps);
        if (rotated < 8 && j < n && !(sum < finite))
            turn_again<DT, INTER>(xb + j * x_step, oa, ob, rotated, p, q, pc, qs, qc, ps);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            p[k] = f2_mul(p[k], r2);
            q[k] = f2_mul(q[k], r2);
        }
        if (j < n) store_pairs<DT, INTER>(yb + j * y_step, oa, ob, p, q);
    }
    griddep_launch_dependents();
}

// The backward on the same rows: persistent, so that a lane, which owns the same
// columns of every head, adds its share of dgamma up in registers; each block
// writes one row of partials per set for the fixed-order column reduce. The sets are
// done one after the other, so that one set's sums and weight are held at a time.
// A group takes a run of up to 8 of a token's heads, for which the cosines and sines are
// computed once (runs of 4: 99 us, of 16: 95.5, against 94); as soon as a head's words are widened, the loads of the head BATCH further on
// take their registers.
// With u = v * g and xr = x * r: mean(u * n) = r * sum(u * x) / D, dgamma += v * xr, and
// dx = r * u - xr * mean(u * n) * r.
template <int DT, bool INTER, int L>
__global__ void __maxnreg__((DT == kF32 ? 168 : 144)) rope_bwd_octets(const RopeArgs a) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    constexpr int BATCH = 2;
    extern __shared__ float sums[];  // [groups of the block][D]
    __shared__ Turns turns;
    const int li = threadIdx.x % L;
    const int groups = blockDim.x / L;
    const int group = threadIdx.x / L;
    griddep_wait();
    int oa, ob;
    lane_octets<INTER>(li, a.D, a.R, oa, ob);
    const int rotated = rotated_pairs(a, li);
    turns.fill(a, L);
    __syncthreads();
    const float inv_d = 1.0f / static_cast<float>(a.D);
#pragma unroll 1
    for (int i = 0; i < a.nsets; ++i) {
        const RopeSet& set = a.set[i];
        const bool norm = set.gamma != nullptr;
        uint64_t gp[4], gq[4], ap[4], aq[4];
        load_gains<DT, INTER>(set, a.one, oa, ob, gp, gq);
#pragma unroll
        for (int k = 0; k < 4; ++k) ap[k] = aq[k] = f2_pack(0.f, 0.f);
        const int run = min(a.chunk, set.heads);
        const int nchunk = (set.heads + run - 1) / run;
        const int64_t items = a.T * nchunk;
        const int64_t d_step = set.dy_head * EB, x_step = set.x_head * EB, y_step = set.y_head * EB;
        for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < items;
             base += static_cast<int64_t>(gridDim.x) * groups) {
            const int64_t item = base + group;
            const bool live = item < items;
            int chunk;
            const int64_t token = split_item(live ? item : 0, nchunk, chunk);
            const int from = chunk * run;
            const int n = live ? min(run, set.heads - from) : 0;
            const int64_t pos = a.pos[token];
            const char* db = static_cast<const char*>(set.dy) + (token * set.dy_token + from * set.dy_head) * EB;
            const char* xb = static_cast<const char*>(set.x) + (token * set.x_token + from * set.x_head) * EB;
            char* yb = static_cast<char*>(set.y) + (token * set.y_token + from * set.y_head) * EB;
            uint32_t dw[BATCH][2][W], xw[BATCH][2][W];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                load16<DT>(db, oa, ob, j < n, dw[j]);
                load16<DT>(xb, oa, ob, norm && j < n, xw[j]);
                db += d_step;
                xb += x_step;
            }
            uint64_t c[4], sn[4], ns[4];
            turns.of_lane(a, li, pos, c, sn);
#pragma unroll
            for (int k = 0; k < 4; ++k) ns[k] = f2_neg(sn[k]);
            // run is the same everywhere: the whole warp goes round as often (the sums see it)
            for (int h = 0; h < run; h += BATCH) {
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    uint64_t p[4], q[4], xp[4], xq[4];
                    to_pairs<DT, INTER>(dw[j], p, q);
                    to_pairs<DT, INTER>(xw[j], xp, xq);
                    const bool more = h + j + BATCH < n;
                    load16<DT>(db, oa, ob, more, dw[j]);
                    load16<DT>(xb, oa, ob, norm && more, xw[j]);
                    db += d_step;
                    xb += x_step;
                    if constexpr (DT == kF32) turn_first_pairs<INTER>(rotated, p, q, c, sn, c, ns);
                    else turn_pairs(p, q, c, sn, c, ns);
                    const bool some = DT != kF32 && rotated < 8 && h + j < n;
                    if (!norm) {
                        uint64_t all = f2_add(p[0], q[0]);
#pragma unroll
                        for (int k = 1; k < 4; ++k) all = f2_add(all, f2_add(p[k], q[k]));
                        const float u = f2_sum(all);
                        if (some && u != u)
                            turn_again<DT, INTER>(db - (BATCH + 1) * d_step, oa, ob, rotated, p, q, c, sn, c, ns);
                    } else {
                        uint64_t ss = f2_pack(0.f, 0.f), ux = f2_pack(0.f, 0.f);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            ss = f2_fma(xq[k], xq[k], f2_fma(xp[k], xp[k], ss));
                            ux = f2_fma(f2_mul(q[k], gq[k]), xq[k], f2_fma(f2_mul(p[k], gp[k]), xp[k], ux));
                        }
                        const float u = f2_sum(ux);
                        if (some && u != u)
                            turn_again<DT, INTER>(db - (BATCH + 1) * d_step, oa, ob, rotated, p, q, c, sn, c, ns);
                        const float r = row_rsqrt(row_sum<L>(f2_sum(ss), nullptr), inv_d, a.eps);
                        const float m = row_sum<L>(u, nullptr) * inv_d * r;
                        const float e = -(r * m);
                        const uint64_t r2 = f2_pack(r, r), e2 = f2_pack(e, e);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            xp[k] = f2_mul(xp[k], r2);
                            xq[k] = f2_mul(xq[k], r2);
                            ap[k] = f2_fma(p[k], xp[k], ap[k]);
                            aq[k] = f2_fma(q[k], xq[k], aq[k]);
                            p[k] = f2_fma(xp[k], e2, f2_mul(f2_mul(p[k], gp[k]), r2));
                            q[k] = f2_fma(xq[k], e2, f2_mul(f2_mul(q[k], gq[k]), r2));
                        }
                    }
                    if (h + j < n) store_pairs<DT, INTER>(yb, oa, ob, p, q);
                    yb += y_step;
                }
            }
        }
        if (!norm) continue;
        __syncthreads();
        // the lane's columns: its octets' entries, in the pairs' order
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float p0, p1, q0, q1;
            f2_unpack(ap[k], p0, p1);
            f2_unpack(aq[k], q0, q1);
            float* row = sums + group * a.D;
            if (INTER) {
                const int o = k < 2 ? oa : ob;
                if (o >= 0) {
                    float* w = row + 8 * o + 4 * (k & 1);
                    w[0] = p0;
                    w[1] = q0;
                    w[2] = p1;
                    w[3] = q1;
                }
            } else {
                if (oa >= 0) {
                    row[8 * oa + 2 * k] = p0;
                    row[8 * oa + 2 * k + 1] = p1;
                }
                if (ob >= 0) {
                    row[8 * ob + 2 * k] = q0;
                    row[8 * ob + 2 * k + 1] = q1;
                }
            }
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

// Halves whose octets do not meet octets (R / 2 no multiple of 8), D whole octets: a lane
// owns octets li and li + L as they stand and gets the entries' partners through shared
// memory. A warp's entry e of octet h * L + li lies at [e][h][lane], so that a lane's
// writes, and the reads at a fixed distance in the row, touch every bank once. Entries from
// R on read a zero. Bound by instructions and, backward, by latency at 12 warps an SM.
// Against entry by entry: bf16 32768 x 40 x 128 with 24 rotated 113 us and 231, its
// backward at 16384 x 20 x 128 66 and 166; 256 with 250 rotated 69 and 143, 113 and 275;
// 512 x 40 x 128 6.0 and 6.6.
constexpr int kSwapFloats = 8 * 2 * 32 + 8;  // of a warp, and the zero

template <int L> struct Swap {
    float* buf;    // this warp's two buffers: heads alternate, with one warp barrier each
    int from[16];  // where the entries' partners lie
    __device__ __forceinline__ Swap(float* all, const RopeArgs& a, int li) {
        const int lane = threadIdx.x & 31;
        buf = all + (threadIdx.x >> 5) * 2 * kSwapFloats;
        if (lane < 2) buf[lane * kSwapFloats + kSwapFloats - 8] = 0.f;
        const int half = a.R / 2;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int col = column(k, li);
            const int to = col < half ? col + half : col - half;
            const int o = to >> 3;
            from[k] = col < a.R ? (to & 7) * 64 + (o / L) * 32 + lane / L * L + o % L : kSwapFloats - 8;
        }
        __syncwarp();
    }
    // The column of a lane's entry k.
    __device__ __forceinline__ static int column(int k, int li) { return 8 * ((k >> 3) * L + li) + (k & 7); }
    // The partners of a lane's entries; `which`: not the buffer of the call before.
    __device__ __forceinline__ void partners(int which, const uint64_t (&f)[8], uint64_t (&p)[8]) const {
        float* b = buf + which * kSwapFloats;
        float* mine = b + (threadIdx.x & 31);
#pragma unroll
        for (int k = 0; k < 8; ++k) f2_unpack(f[k], mine[(2 * k % 8) * 64 + k / 4 * 32], mine[(2 * k % 8 + 1) * 64 + k / 4 * 32]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = f2_pack(b[from[2 * k]], b[from[2 * k + 1]]);
    }
    // An entry is itself * c + its partner * s (back: turned back). Each angle is computed
    // once: a lane has those of pairs 8 li to 8 li + 7, which are its octet's in the first
    // half, and the second half gets them as it gets partners.
    __device__ __forceinline__ void turns(const Turns& turns, const RopeArgs& a, int li, int64_t pos, bool back, uint64_t (&c)[8],
                                          uint64_t (&s)[8]) const {
        uint64_t c4[4], s4[4];
        turns.of_lane(a, li, pos, c4, s4);
        float cs[8], sn[8];
        float* mine = buf + (threadIdx.x & 31);
        __syncwarp();  // the last head's partners have been read
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f2_unpack(c4[k], cs[2 * k], cs[2 * k + 1]);
            f2_unpack(s4[k], sn[2 * k], sn[2 * k + 1]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            mine[k * 64] = cs[k];
            mine[k * 64 + kSwapFloats] = sn[k];
        }
        __syncwarp();
        float ck[16], sk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int col = column(k, li);
            ck[k] = col < a.R ? buf[from[k]] : 1.f;
            sk[k] = buf[from[k] + kSwapFloats];  // 0 from R on
            if (k < 8 && col < a.R / 2) {
                ck[k] = cs[k];
                sk[k] = -sn[k];
            }
            if (back) sk[k] = -sk[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            c[k] = f2_pack(ck[2 * k], ck[2 * k + 1]);
            s[k] = f2_pack(sk[2 * k], sk[2 * k + 1]);
        }
        __syncwarp();
    }
};

template <int DT>
__device__ __forceinline__ void to_entries(const uint32_t (&w)[2][Oct<DT>::kWords], uint64_t (&f)[8]) {
    octet_pairs<DT>(w[0], *reinterpret_cast<uint64_t(*)[4]>(&f[0]));
    octet_pairs<DT>(w[1], *reinterpret_cast<uint64_t(*)[4]>(&f[4]));
}
template <int DT>
__device__ __forceinline__ void store_entries(char* row, int a, int b, const uint64_t (&f)[8]) {
    constexpr int EB = Elem<DT>::kBytes, B = Oct<DT>::kBytes;
    uint32_t w[Oct<DT>::kWords];
    pairs_octet<DT>(*reinterpret_cast<const uint64_t(*)[4]>(&f[0]), w);
    octet_store<EB, Oct<DT>::kWords, true>(row + a * B, w, a >= 0 ? B : 0, false, false);
    pairs_octet<DT>(*reinterpret_cast<const uint64_t(*)[4]>(&f[4]), w);
    octet_store<EB, Oct<DT>::kWords, true>(row + b * B, w, b >= 0 ? B : 0, false, false);
}
template <int DT>
__device__ __forceinline__ void entry_gains(const RopeSet& set, float one, int oa, int ob, uint64_t (&g)[8]) {
    uint32_t w[2][Oct<DT>::kWords];
    load16<DT>(static_cast<const char*>(set.gamma), oa, ob, set.gamma != nullptr, w);
    to_entries<DT>(w, g);
    const float add = set.gamma ? one : 1.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = f2_add(g[k], f2_pack(add, add));
}

// As rope_fwd_octets, but with a run of heads as in rope_bwd_octets: a lane has twice the
// cosines and sines to get.
template <int DT, int L>
__global__ void __maxnreg__(128) rope_fwd_swap(const RopeArgs a) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    constexpr int BATCH = rope_fwd_batch(DT);
    __shared__ Turns turns;
    __shared__ float swaps[kFusedGroupThreads / 32 * 2 * kSwapFloats];
    const int li = threadIdx.x % L;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x / L) + threadIdx.x / L;
    griddep_wait();
    const bool live = item < a.T * a.nchunk;
    int chunk;
    const int64_t token = split_item(live ? item : 0, a.nchunk, chunk);
    const int which = chunk >= a.chunks0 ? 1 : 0;
    if (which) chunk -= a.chunks0;
    const RopeSet& set = a.set[which];
    const int from = chunk * a.chunk;
    const int n = live ? min(a.chunk, set.heads - from) : 0;
    const int oa = li < a.D / 8 ? li : -1, ob = li + L < a.D / 8 ? li + L : -1;
    const char* xb = static_cast<const char*>(set.x) + (token * set.x_token + from * set.x_head) * EB;
    char* yb = static_cast<char*>(set.y) + (token * set.y_token + from * set.y_head) * EB;
    const int64_t x_step = set.x_head * EB, y_step = set.y_head * EB;
    uint32_t xw[BATCH][2][W];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
        load16<DT>(xb, oa, ob, j < n, xw[j]);
        xb += x_step;
    }
    uint64_t c[8], s[8];
    const int64_t pos = a.pos[token];
    const Swap<L> swap(swaps, a, li);
    turns.fill(a, L);
    __syncthreads();
    swap.turns(turns, a, li, pos, false, c, s);
    {
        uint64_t g[8], gp[8];
        entry_gains<DT>(set, a.one, oa, ob, g);
        swap.partners(1, g, gp);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            c[k] = f2_mul(c[k], g[k]);
            s[k] = f2_mul(s[k], gp[k]);
        }
    }
    const float inv_d = 1.0f / static_cast<float>(a.D);
    for (int h = 0; h < a.chunk; h += BATCH) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (h + j >= a.chunk) break;
            uint64_t x[8], p[8];
            to_entries<DT>(xw[j], x);
            load16<DT>(xb, oa, ob, h + j + BATCH < n, xw[j]);
            xb += x_step;
            swap.partners(j & 1, x, p);
            uint64_t ss = f2_mul(x[0], x[0]);
#pragma unroll
            for (int k = 1; k < 8; ++k) ss = f2_fma(x[k], x[k], ss);
            float r = row_rsqrt(row_sum<L>(f2_sum(ss), nullptr), inv_d, a.eps);
            if (!set.gamma) r = 1.f;
            const uint64_t r2 = f2_pack(r, r);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = f2_mul(f2_fma(x[k], c[k], f2_mul(p[k], s[k])), r2);
            if (h + j < n) store_entries<DT>(yb, oa, ob, x);
            yb += y_step;
        }
    }
    griddep_launch_dependents();
}

// As rope_bwd_octets.
template <int DT, int L>
__global__ void __maxnreg__(168) rope_bwd_swap(const RopeArgs a) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    extern __shared__ float sums[];  // [groups of the block][D]
    __shared__ Turns turns;
    __shared__ float swaps[kFusedGroupThreads / 32 * 2 * kSwapFloats];
    const int li = threadIdx.x % L;
    const int groups = blockDim.x / L;
    const int group = threadIdx.x / L;
    griddep_wait();
    const int oa = li < a.D / 8 ? li : -1, ob = li + L < a.D / 8 ? li + L : -1;
    const Swap<L> swap(swaps, a, li);
    turns.fill(a, L);
    __syncthreads();
    const float inv_d = 1.0f / static_cast<float>(a.D);
#pragma unroll 1
    for (int i = 0; i < a.nsets; ++i) {
        const RopeSet& set = a.set[i];
        const bool norm = set.gamma != nullptr;
        uint64_t g[8], acc[8];
        entry_gains<DT>(set, a.one, oa, ob, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = f2_pack(0.f, 0.f);
        const int run = min(a.chunk, set.heads);
        const int nchunk = (set.heads + run - 1) / run;
        const int64_t items = a.T * nchunk;
        const int64_t d_step = set.dy_head * EB, x_step = set.x_head * EB, y_step = set.y_head * EB;
        for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < items;
             base += static_cast<int64_t>(gridDim.x) * groups) {
            const int64_t item = base + group;
            const bool live = item < items;
            int chunk;
            const int64_t token = split_item(live ? item : 0, nchunk, chunk);
            const int from = chunk * run;
            const int n = live ? min(run, set.heads - from) : 0;
            const int64_t pos = a.pos[token];
            const char* db = static_cast<const char*>(set.dy) + (token * set.dy_token + from * set.dy_head) * EB;
            const char* xb = static_cast<const char*>(set.x) + (token * set.x_token + from * set.x_head) * EB;
            char* yb = static_cast<char*>(set.y) + (token * set.y_token + from * set.y_head) * EB;
            uint32_t dw[2][W], xw[2][W];
            load16<DT>(db, oa, ob, n > 0, dw);
            load16<DT>(xb, oa, ob, norm && n > 0, xw);
            uint64_t c[8], s[8];
            swap.turns(turns, a, li, pos, true, c, s);
            // run is the same everywhere: the whole warp goes round as often
#pragma unroll 2
            for (int h = 0; h < run; ++h) {
                uint64_t v[8], x[8], p[8];
                to_entries<DT>(dw, v);
                to_entries<DT>(xw, x);
                db += d_step;
                xb += x_step;
                load16<DT>(db, oa, ob, h + 1 < n, dw);
                load16<DT>(xb, oa, ob, norm && h + 1 < n, xw);
                swap.partners(h & 1, v, p);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = f2_fma(v[k], c[k], f2_mul(p[k], s[k]));
                if (norm) {
                    uint64_t ss = f2_pack(0.f, 0.f), ux = f2_pack(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        ss = f2_fma(x[k], x[k], ss);
                        ux = f2_fma(f2_mul(v[k], g[k]), x[k], ux);
                    }
                    const float r = row_rsqrt(row_sum<L>(f2_sum(ss), nullptr), inv_d, a.eps);
                    const float m = row_sum<L>(f2_sum(ux), nullptr) * inv_d * r;
                    const float e = -(r * m);
                    const uint64_t r2 = f2_pack(r, r), e2 = f2_pack(e, e);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        x[k] = f2_mul(x[k], r2);
                        acc[k] = f2_fma(v[k], x[k], acc[k]);
                        v[k] = f2_fma(x[k], e2, f2_mul(f2_mul(v[k], g[k]), r2));
                    }
                }
                if (h < n) store_entries<DT>(yb, oa, ob, v);
                yb += y_step;
            }
        }
        if (!norm) continue;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int o = k < 4 ? oa : ob;
            if (o >= 0) f2_unpack(acc[k], sums[group * a.D + 8 * o + 2 * (k & 3)], sums[group * a.D + 8 * o + 2 * (k & 3) + 1]);
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

// Any D, R and alignment: a group of L lanes takes a chunk of a token's heads, a lane the
// pairs li, li + L, ... (PK of them at most), loaded and stored entry by entry. The
// entries from R on are paired as neighbours and not turned. Bound by the loads' latency
// and instructions. bf16 32768 x 40 x 90 212 us with four pairs a lane (two of 32 lanes 233,
// eight 283), its backward at 16384 x 20 x 90 136 (158, 249), 16384 x 20 x 250 143 and 274.
template <int L, int PK>
__device__ __forceinline__ void lane_pairs(int li, const RopeArgs& a, bool inter, int (&ca)[PK], int (&cb)[PK]) {
    const int half = a.R / 2;
#pragma unroll
    for (int k = 0; k < PK; ++k) {
        const int i = li + L * k;
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

// A sum over a group's lanes, which groups of a warp come to apart where their chunks end.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    const uint32_t lanes = (L == 32 ? 0xffffffffu : (1u << (L & 31)) - 1u) << ((threadIdx.x & 31) / L * L);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(lanes, v, o);
    return v;
}

template <int DT, int L, int PK, bool BWD>
__global__ void __launch_bounds__(kFusedGroupThreads) rope_pairs(const RopeArgs a) {
    constexpr int EB = Elem<DT>::kBytes;
    extern __shared__ float sums[];  // backward: [groups of the block][D]
    const int li = threadIdx.x % L;
    const int group = threadIdx.x / L;
    const int groups = blockDim.x / L;
    griddep_wait();
    int ca[PK], cb[PK];
    lane_pairs<L, PK>(li, a, a.interleaved != 0, ca, cb);
    float acc[BWD ? kRopeMaxSets : 1][2 * PK];
#pragma unroll
    for (int i = 0; i < (BWD ? kRopeMaxSets : 1); ++i)
#pragma unroll
        for (int k = 0; k < 2 * PK; ++k) acc[i][k] = 0.f;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    const int64_t items = a.T * a.nchunk;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * groups + group; item < items;
         item += static_cast<int64_t>(gridDim.x) * groups) {
        int lo;
        const int64_t token = split_item(item, a.nchunk, lo);
        lo *= a.chunk;
        const int hi = min(lo + a.chunk, a.heads);
        const int64_t pos = a.pos[token];
        float c[PK], s[PK];
#pragma unroll
        for (int k = 0; k < PK; k += 2) {
            const int i0 = li + L * k, i1 = i0 + L, half = a.R / 2;
            c[k] = c[k + 1] = 1.f;
            s[k] = s[k + 1] = 0.f;
            if (i0 < half) {
                uint64_t c2, s2;
                turn_pair(phase_at(turns_per_position(a.inv_freq[i0]), pos),
                          i1 < half ? phase_at(turns_per_position(a.inv_freq[i1]), pos) : 0, a.mscale, a.mscale, c2, s2);
                f2_unpack(c2, c[k], c[k + 1]);
                f2_unpack(s2, s[k], s[k + 1]);
            }
            if (BWD) {
                s[k] = -s[k];
                s[k + 1] = -s[k + 1];
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
                    if (BWD && li + L * k < a.R / 2) {
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
                    r = row_rsqrt(group_sum<L>(ss), inv_d, a.eps);
                    if (BWD) m = group_sum<L>(q) * inv_d * r;
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
                        const bool rotated = li + L * k < a.R / 2;
                        o0 = rotated ? z0 * c[k] - z1 * s[k] : z0;
                        o1 = rotated ? z1 * c[k] + z0 * s[k] : z1;
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
                if (ca[k] >= 0) sums[group * a.D + ca[k]] = acc[i][2 * k];
                if (cb[k] >= 0) sums[group * a.D + cb[k]] = acc[i][2 * k + 1];
            }
            __syncthreads();
            float* out = a.ws + (i * a.units + blockIdx.x) * a.ldws;
            for (int col = threadIdx.x; col < a.D; col += blockDim.x) {
                float t = sums[col];
                for (int k = 1; k < groups; ++k) t += sums[k * a.D + col];
                out[col] = t;
            }
        }
    }
    griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
template <int DT, RopeRows ROWS, bool BWD>
static const void* rope_octets_for(int lanes) {
    constexpr bool INTER = ROWS == kRopeNeighbours;
#define RMSNORM_ROPE(L)                                                                              \
    if (lanes == L) {                                                                                \
        if constexpr (ROWS == kRopeSwap && BWD) return reinterpret_cast<const void*>(&rope_bwd_swap<DT, L>); \
        else if constexpr (ROWS == kRopeSwap) return reinterpret_cast<const void*>(&rope_fwd_swap<DT, L>); \
        else if constexpr (BWD) return reinterpret_cast<const void*>(&rope_bwd_octets<DT, INTER, L>); \
        else return reinterpret_cast<const void*>(&rope_fwd_octets<DT, INTER, L>);                   \
    }
    RMSNORM_ROPE(4)
    RMSNORM_ROPE(8)
    RMSNORM_ROPE(16)
    RMSNORM_ROPE(32)
#undef RMSNORM_ROPE
    return nullptr;
}
template <int DT, bool BWD>
static const void* rope_kernel_for(const RopePlan& p) {
    switch (p.rows) {
    case kRopeNeighbours: return rope_octets_for<DT, kRopeNeighbours, BWD>(p.lanes);
    case kRopeHalves: return rope_octets_for<DT, kRopeHalves, BWD>(p.lanes);
    case kRopeSwap: return rope_octets_for<DT, kRopeSwap, BWD>(p.lanes);
    default: break;
    }
    switch (p.lanes) {
    case 8: return reinterpret_cast<const void*>(&rope_pairs<DT, 8, 4, BWD>);
    case 16: return reinterpret_cast<const void*>(&rope_pairs<DT, 16, 4, BWD>);
    default: break;
    }
    return p.pairs <= 4 ? reinterpret_cast<const void*>(&rope_pairs<DT, 32, 4, BWD>)
                        : reinterpret_cast<const void*>(&rope_pairs<DT, 32, 8, BWD>);
}

const void* rope_kernel(const RopePlan& p, bool bwd) {
    switch (p.dtype) {
    case kF32: return bwd ? rope_kernel_for<kF32, true>(p) : rope_kernel_for<kF32, false>(p);
    case kF16: return bwd ? rope_kernel_for<kF16, true>(p) : rope_kernel_for<kF16, false>(p);
    case kBF16: return bwd ? rope_kernel_for<kBF16, true>(p) : rope_kernel_for<kBF16, false>(p);
    default: return nullptr;
    }
}

}  // namespace rmsnorm
