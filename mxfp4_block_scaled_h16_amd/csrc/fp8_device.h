// Device-side building blocks of 8-bit (E4M3) outputs: a block's scale byte, its codes, and maxima over lanes.
#pragma once

#include "mx_device.h"

namespace mx {

// E8M0 byte of a block from the bit pattern of its largest magnitude: the smallest S with
// amax <= 448 * 2^(S - 127); 448 = 1.75 * 2^8, so the exponent less 8, one more above 1.75.
// 0xFF: the block holds a NaN or infinity.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t amax)
{
    if (amax >= 0x7F800000u) return 0xFFu;
    const int s = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(s, 0);
}

// Four values times 2^(127 - S) (exact: a power of two, S <= 247) as E4M3 codes, rounded to nearest
// even by the conversion; the product is at most 448.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
    return (uint32_t)w;
}
// 2^(127 - S), S in [0, 247]: exponent field 254 - S
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
// the maximum over the 16 lanes of a row, in each of them
__device__ __forceinline__ uint32_t row16_max(uint32_t v)
{
    v = max(v, dpp<0xB1>(v));    // quad_perm [1,0,3,2]
    v = max(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
    v = max(v, dpp<0x141>(v));   // row_half_mirror
    return max(v, dpp<0x140>(v));  // row_mirror
}

// rows that are aligned to their elements only: the 16-byte loads then go to any even address, which
// gfx950 serves (unaligned access is on for every HIP process), at up to twice the lines a load
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

}  // namespace mx
