// octet.cuh -- rows in blocks of 8 columns ("octets"): loads and stores at any
// alignment, conversion, and the counter-based random numbers of the dropout.
//
// The fused kernels (add.cu, quant.cu, rope.cu) give a thread whole octets: 16
// bytes of a 2-byte type, 32 of fp32, 8 of an 8-bit output. One Philox call
// yields eight 16-bit numbers, so an octet is also one call. Rows that do not
// start on a 16-byte boundary are still moved in 16-byte words: a load takes the
// aligned words around the octet and shifts them together, a store takes the
// bytes that share its first aligned word from the previous lane.
#pragma once

#include "device.cuh"

namespace rmsnorm {

// An octet as 32-bit words, and as eight fp32 values.
template <int DT> struct Oct {
    static constexpr int kWords = DT == kF32 ? 8 : 4;
    static constexpr int kBytes = 4 * kWords;
    __device__ __forceinline__ static void unpack(const uint32_t (&w)[kWords], float (&f)[8]) {
        if constexpr (DT == kF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        } else {
            Elem<DT>::unpack(make_uint4(w[0], w[1], w[2], w[3]), f);
        }
    }
    __device__ __forceinline__ static void pack(const float (&f)[8], uint32_t (&w)[kWords]) {
        if constexpr (DT == kF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = Elem<DT>::pack2(f[2 * i], f[2 * i + 1]);
        }
    }
};

// Elements of octet `o` that lie in a row of N.
__device__ __forceinline__ int octet_valid(int o, int N) {
    const int left = N - 8 * o;
    return left < 0 ? 0 : (left > 8 ? 8 : left);
}

// Zero the elements from `valid` on.
template <int DT>
__device__ __forceinline__ void octet_mask(uint32_t (&w)[Oct<DT>::kWords], int valid) {
#pragma unroll
    for (int i = 0; i < Oct<DT>::kWords; ++i) {
        if constexpr (DT == kF32) {
            if (i >= valid) w[i] = 0u;
        } else {
            if (2 * i >= valid) w[i] = 0u;
            else if (2 * i + 1 >= valid) w[i] &= 0xffffu;
        }
    }
}

// Words of the octet at `p` (its first element), of which `valid` elements are
// the row's; the others read as zero. ALIGNED: p is a multiple of 16 and valid is
// 8. Otherwise every 16-byte word that is read holds at least one byte of a valid
// element, so no read leaves the 16-byte words of the tensor.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void octet_load(const char* p, int valid, uint32_t (&w)[Oct<DT>::kWords]) {
    constexpr int W = Oct<DT>::kWords;
    if constexpr (ALIGNED) {
#pragma unroll
        for (int c = 0; c < W / 4; ++c) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[c];
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
        }
    } else {
        const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
        const int need = static_cast<int>(sh) + valid * Elem<DT>::kBytes;  // bytes from the first aligned word on
        const uint4* q = reinterpret_cast<const uint4*>(p - sh);
        uint32_t s[W + 5];
        s[W + 4] = 0u;
#pragma unroll
        for (int c = 0; c < W / 4 + 1; ++c) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (valid > 0 && need > 16 * c) v = q[c];
            s[4 * c] = v.x; s[4 * c + 1] = v.y; s[4 * c + 2] = v.z; s[4 * c + 3] = v.w;
        }
        if (sh & 8u) {
#pragma unroll
            for (int i = 0; i < W + 3; ++i) s[i] = s[i + 2];
        }
        if (sh & 4u) {
#pragma unroll
            for (int i = 0; i < W + 2; ++i) s[i] = s[i + 1];
        }
        const uint32_t bits = 8u * (sh & 3u);
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(s[i], s[i + 1], bits);
        if (valid < 8) octet_mask<DT>(w, valid);
    }
}

// Bytes [from, to) of the `words` aligned words at p; ELEM: bytes of an element
// (from and to are multiples of it).
template <int ELEM, int WORDS>
__device__ __forceinline__ void store_part(char* p, const uint32_t* w, int from, int to) {
#pragma unroll
    for (int j = 0; j < WORDS; ++j) {
        if (from <= 4 * j && to >= 4 * j + 4) {
            reinterpret_cast<uint32_t*>(p)[j] = w[j];
        } else if constexpr (ELEM == 2) {
            if (from <= 4 * j && to >= 4 * j + 2) reinterpret_cast<uint16_t*>(p)[2 * j] = static_cast<uint16_t>(w[j]);
            if (from <= 4 * j + 2 && to >= 4 * j + 4)
                reinterpret_cast<uint16_t*>(p)[2 * j + 1] = static_cast<uint16_t>(w[j] >> 16);
        } else if constexpr (ELEM == 1) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (from <= 4 * j + b && to > 4 * j + b) p[4 * j + b] = static_cast<char>(w[j] >> (8 * b));
        }
    }
}

template <int WORDS>
__device__ __forceinline__ void store_chunk(char* p, const uint32_t* w) {
    if constexpr (WORDS == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Store an octet of W words at `p`, of which the first `bytes` are the row's (0 for
// a lane without one). ALIGNED: p is a multiple of the vector store and bytes is
// 4 * W or 0. Otherwise all 32 lanes call it together: consecutive lanes hold
// consecutive octets of a row; `first` marks a lane whose predecessor does not,
// `last` one whose successor does not (another row, another warp, the row's end).
// Each lane then stores the aligned words that end in its octet, the bytes before
// its octet coming from the lane before.
template <int ELEM, int W, bool ALIGNED>
__device__ __forceinline__ void octet_store(char* p, const uint32_t (&w)[W], int bytes, bool first, bool last) {
    constexpr int AW = W == 2 ? 2 : 4;  // words of a vector store
    constexpr int A = 4 * AW;
    if constexpr (ALIGNED) {
        if (bytes > 0) {
#pragma unroll
            for (int c = 0; c < W / AW; ++c) store_chunk<AW>(p + A * c, &w[AW * c]);
        }
    } else {
        uint32_t s[AW + W + AW + 1];
#pragma unroll
        for (int j = 0; j < AW; ++j) s[j] = __shfl_up_sync(0xffffffffu, w[W - AW + j], 1);
#pragma unroll
        for (int j = 0; j < W; ++j) s[AW + j] = w[j];
#pragma unroll
        for (int j = 0; j <= AW; ++j) s[AW + W + j] = 0u;
        if (bytes <= 0) return;
        const int sh = static_cast<int>(reinterpret_cast<uintptr_t>(p) & (A - 1));
        // out: the words from the aligned address p - sh on
        const int d = A - sh;  // bytes of the predecessor's last A that come before them (A: none of them is needed)
        if (AW == 4 && (d & 8)) {
#pragma unroll
            for (int i = 0; i < AW + W + AW - 1; ++i) s[i] = s[i + 2];
        }
        if (d & 4) {
#pragma unroll
            for (int i = 0; i < AW + W + AW - 1; ++i) s[i] = s[i + 1];
        }
        if (d & A) {
#pragma unroll
            for (int i = 0; i < W + AW; ++i) s[i] = s[i + AW];
        }
        const uint32_t bits = 8u * (static_cast<uint32_t>(d) & 3u);
#pragma unroll
        for (int i = 0; i < W + AW; ++i) s[i] = __funnelshift_r(s[i], s[i + 1], bits);
        const int from = first ? sh : 0;
        const int to = last ? sh + bytes : 4 * W;
        char* base = p - sh;
#pragma unroll
        for (int c = 0; c <= W / AW; ++c) {
            const int lo = from > A * c ? from - A * c : 0;
            const int hi = to < A * (c + 1) ? to - A * c : A;
            if (lo == 0 && hi == A) store_chunk<AW>(base + A * c, &s[AW * c]);
            else if (lo < hi) store_part<ELEM, AW>(base + A * c, &s[AW * c], lo, hi);
        }
    }
}

// ---------------------------------------------------------------------------
// dropout: Philox4x32 with 10 rounds (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011). Counter {octet, row, offset low,
// offset high}, key = seed; the four words' low and high halves, in order, are the
// octet's eight 16-bit numbers. 16 bits per element halve the rounds per element
// against one word each: p is a multiple of 2^-16, and the scale that the kept
// elements get is the inverse of exactly that share.
// ---------------------------------------------------------------------------
struct Dropout {
    const unsigned long long* rng;  // {seed, offset} in device memory
    uint32_t threshold;             // an element is dropped when its number is below; 0: no dropout
    float scale;                    // 65536 / (65536 - threshold)
};

struct PhiloxKey {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ PhiloxKey philox_key(const Dropout& d) {
    const unsigned long long seed = d.rng[0], off = d.rng[1];
    return {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(off),
            static_cast<uint32_t>(off >> 32)};
}

__device__ __forceinline__ void philox_octet(const PhiloxKey& key, uint32_t octet, uint32_t row, uint32_t (&c)[4]) {
    c[0] = octet; c[1] = row; c[2] = key.o0; c[3] = key.o1;
    uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = static_cast<uint64_t>(c[0]) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
        c[0] = static_cast<uint32_t>(b >> 32) ^ c[1] ^ k0;
        c[2] = static_cast<uint32_t>(a >> 32) ^ c[3] ^ k1;
        c[1] = static_cast<uint32_t>(b);
        c[3] = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// f scaled where its number keeps it, 0 (whatever f was) where it is dropped.
__device__ __forceinline__ void dropout_octet(const Dropout& d, const PhiloxKey& key, uint32_t octet, uint32_t row,
                                              float (&f)[8]) {
    uint32_t c[4];
    philox_octet(key, octet, row, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t u = (e & 1) ? c[e / 2] >> 16 : c[e / 2] & 0xffffu;
        f[e] = u >= d.threshold ? f[e] * d.scale : 0.f;
    }
}

// ---------------------------------------------------------------------------
// sums over a row's threads. G lanes (a power of two) per row, or, with G == 0,
// the whole block: one barrier, `part` (32 floats) not reused before the next one.
// Every thread of the row gets the same bits.
// ---------------------------------------------------------------------------
template <int G>
__device__ __forceinline__ float row_sum(float v, float* part) {
    if constexpr (G > 0) {
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    } else {
        const int lane = threadIdx.x & 31;
        v = warp_allsum(v);
        if (lane == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        return warp_allsum(lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0.f);
    }
}

}  // namespace rmsnorm
