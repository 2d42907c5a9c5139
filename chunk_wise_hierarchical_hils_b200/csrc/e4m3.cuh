// e4m3.cuh -- conversions between float32 and the e4m3 bytes of the 8-bit cache (sm_100a).
//
// e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; largest value 448, smallest normal 2^-6, subnormals
// down to 2^-9, no infinities, 0x7F / 0xFF is NaN.  Every e4m3 value is exact in f16.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace hils {

constexpr int kScaleExpMin = -100, kScaleExpMax = 119;   // exponents a written scale may have

// Two floats -> two e4m3 bytes (lo in the low byte), nearest even, +-448 beyond the range.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    return to_e4m3x2(a, b) | (to_e4m3x2(c, d) << 16);
}

// Two e4m3 bytes (the low 16 bits of v) -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}

// Four e4m3 bytes -> floats, exact.
__device__ __forceinline__ void e4m3x4_to_float(uint32_t v, float *o)
{
    const uint32_t a = e4m3x2_to_f16x2(v), b = e4m3x2_to_f16x2(v >> 16);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    o[0] = x.x; o[1] = x.y; o[2] = y.x; o[3] = y.y;
}

// Exponent e of a written scale 2^e for a largest magnitude m (finite, >= 0): the smallest e with
// m <= 448 * 2^e = 1.75 * 2^(e + 8), read off m's exponent and fraction, clamped to the range above.
__device__ __forceinline__ int scale_exponent(float m)
{
    const uint32_t u = __float_as_uint(m);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(kScaleExpMin, min(kScaleExpMax, e));
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

}  // namespace hils
