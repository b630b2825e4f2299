// rope.cuh -- the rotation of head rows by position, shared by rope.cu (forward and backward)
// and append.cu (into a paged cache): angles in fixed point, how lanes hold a row's pairs, and
// the turns. The formulas and the reasons for the angles are at the top of rope.cu.
#pragma once

#include "fused.h"
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

}  // namespace rmsnorm
