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

// |y| as an integer: ordered as the value, with NaN above infinity.
__device__ __forceinline__ uint32_t magnitude(float y) { return __float_as_uint(y) & 0x7fffffffu; }

// The largest magnitude of elements [0, valid) of an octet.
__device__ __forceinline__ uint32_t octet_amax(const uint64_t (&y)[4], int valid) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(y[i], a, b);
        m = max(m, 2 * i < valid ? magnitude(a) : 0u);
        m = max(m, 2 * i + 1 < valid ? magnitude(b) : 0u);
    }
    return m;
}

__device__ __forceinline__ float quant_scale(uint32_t amax, int pow2) {
    float s = __uint_as_float(amax) * (1.0f / 448.0f);
    if (s < 1.17549435e-38f) s = 1.17549435e-38f;  // 2^-126; a NaN stays
    if (pow2) {
        // up to the next power of two: a carry out of the fraction raises the exponent
        // (infinity and NaN stay)
        const uint32_t b = __float_as_uint(s);
        if (b < 0x7f800000u) s = __uint_as_float((b + 0x007fffffu) & 0x7f800000u);
    }
    return s;
}

// Codes of octet `o` of a row (`valid` elements of y), and its group's scale from the
// group's largest magnitude, by the group's first octet. Unless ALIGNED every lane of a
// warp calls it (octet_store).
template <bool ALIGNED>
__device__ __forceinline__ void quant_store(const AddArgs& a, int64_t row, int o, int valid, const uint64_t (&y)[4],
                                            uint32_t amax, bool first, bool last) {
    const float s = quant_scale(amax, a.pow2);
    // the scale is a normal number and its inverse too: off by at most 1 unit in the last place
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    uint32_t code[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) code[i] = e4m3_pair(y[2 * i], inv) | e4m3_pair(y[2 * i + 1], inv) << 16;
    if (!ALIGNED || valid > 0)
        octet_store<1, 2, ALIGNED>(static_cast<char*>(a.y) + row * a.ldy + o * 8, code, valid, first, last);
    if (valid > 0) {
        float* sr = a.scales + row * a.ldscales;
        if (a.group == 0) {
            if (o == 0) sr[0] = s;
        } else if (o % (a.group / 8) == 0) {
            sr[o / (a.group / 8)] = s;
        }
    }
}

}  // namespace rmsnorm
