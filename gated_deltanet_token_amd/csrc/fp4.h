// e2m1 codes (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte,
// the first in the low half, and e8m0 scales, on gfx950.
#pragma once

#include "gdn_device.h"

namespace gdn {

constexpr int kScaleBlock = 32;         // elements of a key that share a scale
constexpr int kGranule = 16;            // tokens whose codes of a value's element lie together
constexpr float kLeastScale = 0x1p-100f;

// eight codes of |x| < 7, round to nearest even
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], 1.0f, 3);
}

// the values of eight codes as bf16 pairs, times `scale`, a power of two
__device__ __forceinline__ uint4 e2m1_bf16(uint32_t w, float scale = 1.0f) {
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3)));
}

// The exponent of the scale of a block whose largest magnitude is `amax`
// (finite): that of amax rounded to one bit behind the leading one, ties to even,
// less two, so that amax is met by a code from 3.5 to 7 (7 excluded); -100 at
// least.
__device__ __forceinline__ int e2m1_block_exponent(float amax) {
    const uint32_t u = __builtin_bit_cast(uint32_t, amax);
    const int e = (int)(u >> 23) - 127 - 2 + ((u & 0x7fffffu) >= 0x600000u ? 1 : 0);
    return max(e, -100);                             // subnormal and zero amax too
}

}  // namespace gdn
