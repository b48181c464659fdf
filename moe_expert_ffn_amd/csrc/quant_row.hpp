// The per-token int8 quantisation arithmetic of FrontReorder (step 2c of section
// 1 of the pto-isa MegaMoE overview page), shared by the permute kernels and the
// few-token layer so that both produce the same codes.
#pragma once

#include "common.hpp"

namespace megamoe {

// CAST_ROUND(x / scale) for x an fp16 value of a row whose largest |x| is amax
// (also fp16), scale = amax / 127 and inv = 1 / scale (both IEEE; inv = 0 for
// an all-zero row, which gives 0 everywhere).
//  * The quotient is x * inv corrected once by its FMA residual,
//    q + inv * (x - q * scale) (Markstein's method): three instructions instead
//    of the ten of an IEEE division.  The first product is an FMA with a +0
//    addend so that the hardware reads x as fp16 in the same instruction.
//  * Half away from zero is the truncation of q + copysign(0.49999997, q), the
//    largest float below one half (adding exactly one half would take
//    0.49999997 itself to 1), and the truncation is the float -> int
//    conversion: two instructions and the conversion instead of the six of
//    roundf.  |x| <= amax keeps the sum within (-127.5, 127.5), so no clamp
//    is needed.
// For every finite fp16 amax > 0 and every fp16 x with |x| <= amax this gives
// the same integer as roundf of the IEEE quotient, clamped to [-127, 127];
// tests/csrc/quant_exhaustive.c checks all 1,007,681,535 such pairs.
__device__ __forceinline__ int quant_round(float x, float scale, float inv) {
    const float q0 = __builtin_fmaf(x, inv, 0.0f);
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, scale, x), inv, q0);
    return (int)(q + __builtin_copysignf(0x1.fffffep-2f, q));
}

// 8 fp16 values (one 16-byte word) -> 8 int8 codes.  The low bytes of four
// codes are gathered into a word by three byte permutes.
__device__ __forceinline__ uint2 quant_chunk8(const uint4 &raw, float scale, float inv) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw);
    uint32_t packed[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        int q[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int idx = j * 4 + h;  // element within the 8-element chunk
            const uint16_t bits = (uint16_t)((w[idx >> 1] >> ((idx & 1) * 16)) & 0xffffu);
            q[h] = quant_round(h2f(bits), scale, inv);
        }
        // bytes [q0, q1, 0, 0] and [q2, q3, 0, 0], then [q0, q1, q2, q3]
        const uint32_t lo = __builtin_amdgcn_perm((uint32_t)q[1], (uint32_t)q[0], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm((uint32_t)q[3], (uint32_t)q[2], 0x0c0c0400u);
        packed[j] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
    return make_uint2(packed[0], packed[1]);
}

// The largest |x| over 16-byte words of fp16 values, as fp16 bits.  With the
// sign bits cleared, finite fp16 values order like their bit patterns, so the
// maximum takes one packed 16-bit integer max per two values.  (The
// quantiser's inputs are finite; a NaN would be taken as the maximum.)
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2_t absmax_step(u16x2_t m, const uint4 &raw) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[j] & 0x7fff7fffu));
    return m;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, off, kWave);
        v = o > v ? o : v;
    }
    return v;
}

}  // namespace megamoe
