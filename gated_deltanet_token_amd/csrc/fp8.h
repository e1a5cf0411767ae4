// e4m3 (OCP) codes on gfx950.
#pragma once

#include "gdn_device.h"

namespace gdn {

// four codes from four values, round to nearest even; |x| <= 448, or infinite or
// NaN: NaN (the format has no infinities)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// the values of four codes
__device__ __forceinline__ void e4m3_values(uint32_t w, float (&f)[4]) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    f[0] = lo.x;
    f[1] = lo.y;
    f[2] = hi.x;
    f[3] = hi.y;
}

// four codes of one scale at another: each value times `ratio`, rounded again
__device__ __forceinline__ uint32_t e4m3_rescaled(uint32_t w, float ratio) {
    float f[4];
    e4m3_values(w, f);
    return e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// The scale of a block whose largest magnitude is `amax` (finite): the least
// power of two s >= 2^-100 with amax <= 448 s.  448 = 1.75 * 2^8, so it is
// amax's own power of two over 2^8, twice that where the significand is above
// 1.75.
__device__ __forceinline__ float e4m3_block_scale(float amax) {
    const uint32_t u = __builtin_bit_cast(uint32_t, amax);
    int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);   // biased exponent of s
    e = max(e, 127 - 100);                                                // subnormal and zero amax too
    return __builtin_bit_cast(float, (uint32_t)e << 23);
}

}  // namespace gdn
