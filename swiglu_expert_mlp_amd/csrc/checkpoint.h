// Activations kept in 8 bits: the gate and up values of a grouped row, in blocks of 32
// columns (gate and up by turns, the interleaved order of FC1's columns) that share one
// scale 2^(byte - 127): the smallest power of two, at least 2^-126, whose 127-fold reaches
// the block's largest magnitude.  A code is the value over the scale rounded to the nearest
// integer, ties to even, so no code is beyond +-127 and a value is off by at most half a
// scale: less than 1/127 of its block's largest magnitude, or 2^-127 where the scale is at
// its floor of 2^-126 (a largest magnitude below 127 2^-126).  For near-normal values that
// is 0.74 % of their deviation in the mean, which brings 0.95 to 1.2 % to the gradients.
// (E4M3 codes would be off by 2^-4 of each value: about three times the mean error.  A power
// of two costs up to a bit against amax / 127, and a quarter of the scales' bytes.)
// A block with an infinity or a NaN has byte 255 and codes of 0: its values read back as NaN.
#pragma once

#include "common.h"

namespace moe {

// Scale byte of a block whose magnitudes' bit patterns are at most `amax` (as integers,
// where infinities and NaNs are the largest): amax = 1.m 2^E with 127 = 1.984375 2^6
__device__ __forceinline__ uint32_t ckpt_byte(uint32_t amax)
{
    const int ef = (int)(amax >> 23);
    const int b = ef - 6 + ((amax & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return ef == 255 ? 255u : (uint32_t)(b < 1 ? 1 : b);
}

// 2^(127 - byte), the factor that takes values to codes; 0 for byte 255
__device__ __forceinline__ float ckpt_factor(uint32_t byte)
{
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); 0 for byte 0, infinity for byte 255 (times code 0: NaN)
__device__ __forceinline__ float ckpt_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// The code of v in the low byte: adding 1.5 2^23 leaves the nearest integer, ties to even,
// in the last bits of the sum (two's complement).  Factor 0 with an infinity or a NaN gives
// a NaN pattern, which the caller masks with byte 255.
__device__ __forceinline__ uint32_t ckpt_code(float v, float factor)
{
    return __float_as_uint(__builtin_fmaf(v, factor, 12582912.0f));
}

// The larger of this lane's value and its neighbour's (lane ^ 1)
__device__ __forceinline__ uint32_t pair_max_u32(uint32_t x)
{
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xf, 0xf, false));   // quad_perm [1, 0, 3, 2]
}

}  // namespace moe
