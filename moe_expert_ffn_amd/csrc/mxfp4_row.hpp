// The arithmetic of one MXFP4 block: its scale from the largest |x|, and elements as codes.
#pragma once

#include "common.hpp"

namespace megamoe {

// E8M0 byte -> the fp32 power of two (byte 0 is the subnormal 2^-127; 255 NaN)
__device__ __forceinline__ float e8m0_f32(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x400000u : b == 255 ? 0x7fc00000u : b << 23);
}

// The block's scale byte from the fp32 bits of max|x| (NaN orders above infinity): its biased
// exponent less 2; below 2^-125 the scale stays 2^-127; 255 where the block is not finite.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t m) {
    const uint32_t ex = m >> 23;
    return ex == 255 ? 255 : ex < 2 ? 0 : ex - 2;
}

// The codes of eight elements, the first one lowest.  v_cvt_scalef32_pk_fp4_f32 divides by the scale,
// rounds to nearest even and saturates.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], uint32_t b) {
    if (b == 255) return 0;
    const float s = e8m0_f32(b);
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
}

}  // namespace megamoe
