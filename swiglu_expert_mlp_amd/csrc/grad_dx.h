// The rows of x's gradient between the product that makes them and the sum over a token's
// routes: 16-bit integers, 16 neighbouring columns sharing a scale 2^(byte - 127), the
// smallest power of two (at least 2^-126) whose 32767-fold reaches their largest magnitude.
// A value is off by at most half a scale: less than 1/32767 of that magnitude, or 2^-127 where
// the scale is at its floor (a largest magnitude below 32767 2^-126).  So d_x carries the
// roundings of its operand and its own to bf16 alone, but for values less than 1/128 of the
// loudest of their 16, which keep fewer bits than bf16 rows would leave them.  (bf16 rows would
// add a third rounding to every value; fp32 rows are twice the bytes: at 16K tokens, top-8,
// hidden 2048, the sum took 212 us instead of 117.)
// Where one of the 16 is an infinity or a NaN the byte is 255 and the values are bf16 patterns.
#pragma once

#include "common.h"

namespace moe {

__device__ __forceinline__ uint32_t dx_pack16(const float (&v)[16], uint32_t (&w)[8])
{
    uint32_t amax = 0;
#pragma unroll
    for (int m = 0; m < 16; ++m) amax = max(amax, __float_as_uint(v[m]) & 0x7fffffffu);
    // amax = 1.m 2^E against 32767 = 1.99994 2^14; infinities and NaNs are the largest patterns
    const int ef = (int)(amax >> 23);
    const int b = ef - 14 + ((amax & 0x7fffffu) > 0x7ffe00u ? 1 : 0);
    const uint32_t byte = ef == 255 ? 255u : (uint32_t)(b < 1 ? 1 : b);
    if (__builtin_expect(__any(ef == 255), 0)) {
        if (ef == 255) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
                w[m] = (uint32_t)f32_to_bf16_bits(v[2 * m]) | ((uint32_t)f32_to_bf16_bits(v[2 * m + 1]) << 16);
            return byte;
        }
    }
    // adding 1.5 2^23 leaves the nearest integer, ties to even, in the last 16 bits
    const float f = __uint_as_float((254u - byte) << 23);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const uint32_t lo = __float_as_uint(__builtin_fmaf(v[2 * m], f, 12582912.0f));
        const uint32_t hi = __float_as_uint(__builtin_fmaf(v[2 * m + 1], f, 12582912.0f));
        w[m] = (lo & 0xffffu) | (hi << 16);
    }
    return byte;
}

// Two values of a pair of codes
__device__ __forceinline__ void dx_unpack(uint32_t w, uint32_t byte, float& a, float& b)
{
    const float s = __uint_as_float(byte << 23);
    const bool raw = byte == 255u;
    a = raw ? __uint_as_float(w << 16) : (float)((int)(w << 16) >> 16) * s;
    b = raw ? __uint_as_float(w & 0xffff0000u) : (float)((int)w >> 16) * s;
}

}  // namespace moe
