// The 8-bit cache: e4m3 codes with one power-of-two scale for each block of
// consecutive tokens of one (page, KV head).
//
// A block's scale is the least 2^e (e >= -126) with amax <= 448 * 2^e, 448
// being e4m3's largest value. e4m3 is a floating type, so rounding the scale
// up to a power of two costs range (one binade of 17), not precision, and it
// buys exactness: codes that move to a larger scale when a later token raises
// the block's amax keep their value unless it falls among the subnormals, and
// products with the scale never round.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace loki {

constexpr float kE4m3Max = 448.f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126, the scale of an all-zero block

// The least power of two s >= 2^-126 with amax <= 448 s. 448 = 1.75 * 2^8, so
// with amax = 1.f * 2^x the exponent is x - 8, one more when 1.f > 1.75.
__device__ __forceinline__ float pow2_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased by 127
    e = e < 1 ? 1 : e;
    return __uint_as_float((uint32_t)e << 23);
}

// |x| for the block's amax: infinities and NaN do not count
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

// two fp32 -> two e4m3 (lo in the low byte): nearest even, saturating at 448
// (also infinities); NaN gives NaN
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// two e4m3 (low 16 bits) -> two fp16, exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// four e4m3 -> four fp32, exact
__device__ __forceinline__ void e4m3x4_to_float(uint32_t v, float* f) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(v & 0xffffu));
    const float2 b = f16x2_to_float2(e4m3x2_to_f16x2(v >> 16));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

}  // namespace loki
