// quant.cuh -- e4m3 codes and their scales, of quant.cu.
#pragma once

#include "fused.h"
#include "octet.cuh"

namespace rmsnorm {

// A pair times inv as two e4m3, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(uint64_t y, float inv) {
    float a, b;
    f2_unpack(f2_mul(y, f2_pack(inv, inv)), a, b);
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(b), "f"(a));
    return v;
}

// The larger of a and |b|; a NaN of either stays (fmaxf drops it).
__device__ __forceinline__ float max_magnitude(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
    return m;
}

// The largest magnitude of elements [lo, hi) of an octet.
template <bool ALIGNED>
__device__ __forceinline__ float octet_amax(const uint64_t (&z)[4], int lo, int hi) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(z[i], a, b);
        m = max_magnitude(m, ALIGNED || (2 * i >= lo && 2 * i < hi) ? a : 0.f);
        m = max_magnitude(m, ALIGNED || (2 * i + 1 >= lo && 2 * i + 1 < hi) ? b : 0.f);
    }
    return m;
}

// The scale of a group whose largest |z| is amax, with y = z * r; and the factors by which
// z becomes codes, in this order: 1 and r / scale, the r of y and of the scale having
// cancelled, or, at the least scale and for the smallest z, where that may overflow, r
// and 1 / scale.
__device__ __forceinline__ float quant_scale(float amax, float r, int pow2, float& f0, float& f1) {
    float s = amax * r * (1.0f / 448.0f);
    const bool apart = s < 1.17549435e-38f || amax < 7.8886091e-31f;  // 2^-126 and 2^-100
    if (s < 1.17549435e-38f) s = 1.17549435e-38f;                   // a NaN stays
    if (pow2) {
        // up to the next power of two: a carry out of the fraction raises the exponent
        // (infinity and NaN stay)
        const uint32_t b = __float_as_uint(s);
        if (b < 0x7f800000u) s = __uint_as_float((b + 0x007fffffu) & 0x7f800000u);
    }
    // the scale is a normal number and its inverse too: off by at most 1 unit in the last place
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    f0 = apart ? r : 1.f;
    f1 = apart ? inv : r * inv;
    return s;
}

// Codes of octet `o` of a row, and its group's scale from the group's largest |z|, by
// the group's first octet (groups of columns want octets that start at column 0). Unless ALIGNED every lane of a
// warp calls it (octet_store).
template <bool ALIGNED>
__device__ __forceinline__ void quant_store(const AddArgs& a, int64_t row, int o, const Cut& cut, uint64_t (&z)[4], float amax,
                                            float r, bool first, bool last) {
    if (ALIGNED && !cut.live()) return;
    float f0, f1;
    const float s = quant_scale(amax, r, a.pow2, f0, f1);
    if (f0 != 1.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = f2_mul(z[i], f2_pack(f0, f0));
    }
    uint32_t code[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) code[i] = e4m3_pair(z[2 * i], f1) | e4m3_pair(z[2 * i + 1], f1) << 16;
    octet_store<1, 2, ALIGNED>(static_cast<char*>(a.y) + row * a.ldy + cut.col, code, cut.hi, first, last,
                               first ? cut.lo : (cut.col < 8 ? 8 - cut.col : 0));
    if (cut.live()) {
        float* sr = a.scales + row * a.ldscales;
        if (a.group == 0) {
            if (o == 0) sr[0] = s;
        } else if ((o & ((1 << a.group_shift) - 1)) == 0) {
            sr[o >> a.group_shift] = s;
        }
    }
}

}  // namespace rmsnorm
