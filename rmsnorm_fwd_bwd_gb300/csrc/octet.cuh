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
#include "fused.h"

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

// An octet as four packed pairs of fp32 values (f2_*: one instruction for two).
template <int DT>
__device__ __forceinline__ void octet_pairs(const uint32_t (&w)[Oct<DT>::kWords], uint64_t (&f)[4]) {
    float e[8];
    Oct<DT>::unpack(w, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_pack(e[2 * i], e[2 * i + 1]);
}
template <int DT>
__device__ __forceinline__ void pairs_octet(const uint64_t (&f)[4], uint32_t (&w)[Oct<DT>::kWords]) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(f[i], e[2 * i], e[2 * i + 1]);
    Oct<DT>::pack(e, w);
}

// Keep elements [lo, hi) of an octet, the others become zero.
template <int DT>
__device__ __forceinline__ void octet_keep(uint32_t (&w)[Oct<DT>::kWords], int lo, int hi) {
#pragma unroll
    for (int i = 0; i < Oct<DT>::kWords; ++i) {
        if constexpr (DT == kF32) {
            if (i < lo || i >= hi) w[i] = 0u;
        } else {
            if (2 * i < lo || 2 * i >= hi) w[i] &= 0xffff0000u;
            if (2 * i + 1 < lo || 2 * i + 1 >= hi) w[i] &= 0xffffu;
        }
    }
}

// The octet that starts `sh` bytes (a multiple of the element size, below 16) into the
// words s.
template <int DT>
__device__ __forceinline__ void octet_shift(uint32_t (&s)[Oct<DT>::kWords + 5], uint32_t sh, uint32_t (&w)[Oct<DT>::kWords]) {
    constexpr int W = Oct<DT>::kWords;
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
}

// The octet at `p` (where its first element is or would be), of which elements
// [lo, hi) are the row's; the others read as zero. ALIGNED: p is a multiple of 16, lo
// is 0 and hi 8. Otherwise every 16-byte word that is read holds at least one byte of
// one of the elements, so no read leaves the 16-byte words of the tensor.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void octet_load(const char* p, int lo, int hi, uint32_t (&w)[Oct<DT>::kWords]) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    if constexpr (ALIGNED) {
#pragma unroll
        for (int c = 0; c < W / 4; ++c) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[c];
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
        }
    } else {
        const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
        const int from = static_cast<int>(sh) + lo * EB, to = static_cast<int>(sh) + hi * EB;  // bytes after p - sh
        const uint4* q = reinterpret_cast<const uint4*>(p - sh);
        uint32_t s[W + 5];
        s[W + 4] = 0u;
#pragma unroll
        for (int c = 0; c < W / 4 + 1; ++c) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (from < 16 * c + 16 && to > 16 * c) v = q[c];
            s[4 * c] = v.x; s[4 * c + 1] = v.y; s[4 * c + 2] = v.z; s[4 * c + 3] = v.w;
        }
        if (sh != 0u) {
            octet_shift<DT>(s, sh, w);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = s[i];
        }
        if (lo > 0 || hi < 8) octet_keep<DT>(w, lo, hi);
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

// Store an octet of W words at `p`, of which the bytes up to `bytes` are the row's (0 for
// a lane without one). `skip`: the bytes before the row's start in the octet, or, for a
// lane that is not `first`, in the octet before. ALIGNED: p is a multiple of the vector
// store, bytes is 4 * W or 0 and skip 0. Otherwise all 32 lanes call it together: consecutive lanes hold
// consecutive octets of a row; `first` marks a lane whose predecessor does not,
// `last` one whose successor does not (another row, another warp, the row's end).
// Each lane then stores the aligned words that end in its octet, the bytes before
// its octet coming from the lane before.
template <int ELEM, int W, bool ALIGNED>
__device__ __forceinline__ void octet_store(char* p, const uint32_t (&w)[W], int bytes, bool first, bool last, int skip = 0) {
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
        const int from = first ? sh + skip : (sh + skip > 4 * W ? sh + skip - 4 * W : 0);
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

// Load an octet of a row: whole 16-byte words (and the ends masked), or octet_load.
template <int DT, int MODE>
__device__ __forceinline__ void row_load(const char* p, int lo, int hi, uint32_t (&w)[Oct<DT>::kWords]) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    if constexpr (MODE == kRowsOnePhase) {
#pragma unroll
        for (int c = 0; c < W / 4; ++c) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (W == 4 || (lo * EB < 16 * c + 16 && hi * EB > 16 * c)) v = reinterpret_cast<const uint4*>(p)[c];
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
        }
        if (lo > 0 || hi < 8) octet_keep<DT>(w, lo, hi);
    } else {
        octet_load<DT, MODE == kRowsAligned>(p, lo, hi, w);
    }
}

// Store an octet at p, of which elements [lo, hi) are the row's. ALIGNED as above.
// on_word: p is a multiple of 16 (the octets follow this tensor's rows); else octet_store,
// called by the whole warp, with lo 0.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void octet_put(char* p, const uint32_t (&w)[Oct<DT>::kWords], int lo, int hi, bool on_word,
                                          bool first, bool last) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    if (ALIGNED || on_word) {
        if (ALIGNED ? hi > 0 : lo == 0 && hi == 8) {
#pragma unroll
            for (int c = 0; c < W / 4; ++c) store_chunk<4>(p + 16 * c, &w[4 * c]);
        } else if (hi > lo) {
            store_part<EB, W>(p, w, lo * EB, hi * EB);
        }
    } else {
        octet_store<EB, W, false>(p, w, hi > 0 ? hi * EB : 0, first, last);
    }
}

// How a row is cut into octets. They start at the columns 8 * o - phase, phase being
// the elements that the outputs' row starts after a 16-byte boundary (0 for aligned
// rows): the outputs, and the inputs that share the offset, then move in whole
// 16-byte words, and only a row's two ends are masked.
struct Cut {
    int col, lo, hi;  // first column, and the octet's elements in the row
    __device__ __forceinline__ Cut() {}
    __device__ __forceinline__ Cut(int o, int phase, int N) {
        col = 8 * o - phase;
        lo = col < 0 ? -col : 0;
        const int left = N - col;
        hi = left < 0 ? 0 : (left > 8 ? 8 : left);
    }
    __device__ __forceinline__ bool live() const { return hi > 0; }
};

// Aligned rows: octets are whole or missing.
__device__ __forceinline__ Cut whole_cut(int o, int N) {
    Cut c;
    c.col = 8 * o;
    c.lo = 0;
    c.hi = c.col < N ? 8 : 0;
    return c;
}

// The elements that p starts after a 16-byte boundary.
template <int DT> __device__ __forceinline__ int word_phase(const void* p) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / Elem<DT>::kBytes);
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
    // A number in the upper half of a word is at least the threshold where the word is
    // above this, whatever its lower half (with a threshold of 65536: nowhere).
    __device__ __forceinline__ uint32_t below() const { return (threshold << 16) - 1u; }
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
    // opaque, so that the rounds' keys are added up here: hoisted out of a loop over
    // rows they would hold 20 registers
    asm volatile("" : "+r"(k0), "+r"(k1));
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

// The octet whose first column is col: f scaled where its number keeps it, 0 (whatever f
// was) where it is dropped. ANY: the octet may start inside a counter's eight columns,
// and takes two calls then.
template <bool ANY>
__device__ __forceinline__ void dropout_octet(const Dropout& d, const PhiloxKey& key, int col, uint32_t row, uint64_t (&f)[4]) {
    uint32_t s[9];
    {
        uint32_t c[4];
        philox_octet(key, static_cast<uint32_t>(col >> 3), row, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = c[i];
    }
    if (ANY && (col & 7) != 0) {
        uint32_t c[4];
        philox_octet(key, static_cast<uint32_t>((col >> 3) + 1), row, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 + i] = c[i];
        s[8] = 0u;
        if (col & 4) {
#pragma unroll
            for (int i = 0; i < 7; ++i) s[i] = s[i + 2];
        }
        if (col & 2) {
#pragma unroll
            for (int i = 0; i < 6; ++i) s[i] = s[i + 1];
        }
        const uint32_t bits = (col & 1) ? 16u : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = __funnelshift_r(s[i], s[i + 1], bits);
    }
    const uint32_t below = d.below();
    const uint64_t scale = f2_pack(d.scale, d.scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(f2_mul(f[i], scale), lo, hi);
        f[i] = f2_pack((s[i] << 16) > below ? lo : 0.f, s[i] > below ? hi : 0.f);
    }
}

// ---------------------------------------------------------------------------
// sums over a row's threads. G lanes (a power of two) per row, or, with G == 0,
// the whole block: one barrier, `part` (32 floats) not reused before the next one.
// Every thread of the row gets the same bits.
// ---------------------------------------------------------------------------
// The largest of the 32 lanes' non-negative values, a NaN before any number. By shuffles:
// behind a branch that not all lanes take, __reduce_max_sync was seen to be run by the
// two sides apart (nvcc 13.0).
__device__ __forceinline__ float warp_allmax(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(w));
    }
    return v;
}

// 1 / sqrt(sum / N + eps) for head rows and for the scales of the 8-bit output (whose codes it
// cancels from): rsqrtf is off by at most 2 units in the last place, and the IEEE root and
// quotients would cost some forty instructions per thread and row.
__device__ __forceinline__ float row_rsqrt(float sum, float inv_n, float eps) { return rsqrtf(fmaf(sum, inv_n, eps)); }

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
